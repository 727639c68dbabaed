"""The mixture-of-experts calls on the GPU against the fp64 CPU oracle (oracle/experts.py).

Tolerances, from the arithmetic of include/dlc.h and u = 2^-24.  Of a probability: its exponent's argument is
(x - m) log2(e), two roundings and the constant's, 2.3 u per unit of x - m after the exponential, itself 2 u; the
same for the row's sum, whose at most 22 additions add u each; the reciprocal 2 u and two products.  With D the
row's largest distance from its maximum that a probability above 2^-126 has, R(D) = (4.6 D + 31) u in all.
  * means: R, 15 additions, the rounding to fp32;  loss: a sum of positive terms: R, 15 additions and one more;
  * the gradient p (c - sum p c): with A the largest |c|, p A (3 R + 64 u), then the type's rounding, eps / 2 of the
    value or half its smallest subnormal;
  * counts, totals, merge weights and the step: the same operations in the same order: equal;
  * the norm: fp64 sums in some order: relative 2^-40.
"""
import numpy as np
import pytest
import torch

import diloco_outer_step_amd as dlc
from oracle import experts

pytestmark = pytest.mark.gpu

DEV = "cuda"
U = 2.0 ** -24
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
TINY = {"fp32": 2.0 ** -126, "bf16": 2.0 ** -126, "fp16": 2.0 ** -25}
SENT = 77.0


def widen(t):
    return t.double().cpu().numpy()


class Router:
    """Inputs of one call in padded buffers full of sentinels, the call, and its comparison with the oracle."""

    def __init__(self, k, t, e, top, kind="fp32", ids=torch.int64, masked=False, pad=0, seed=0, skew=1.0, first=0):
        g = torch.Generator().manual_seed(seed)
        self.k, self.t, self.e, self.top, self.kind = k, t, e, top, kind
        shape = (k, t + 1, e + pad + first)

        def inner(b):  # the call's part of a buffer: padded rows, another row behind the last token
            return b[:, :t, first:first + e]

        x = torch.randn(shape, generator=g) * 2 + skew * torch.randn((k, 1, shape[2]), generator=g)
        self.x_all = x.to(TYPES[kind]).to(DEV)
        self.x = inner(self.x_all)
        best = torch.topk(self.x.float().cpu(), top, dim=-1)[1]
        self.ids_all = torch.full((k, t + 1, top + 3), -5, dtype=ids)
        self.ids_all[:, :t, :top] = best.to(ids)
        self.ids_all = self.ids_all.to(DEV)
        self.ids = self.ids_all[:, :t, :top]
        self.mask = None
        if masked:
            self.mask = (torch.rand((k, t + 5), generator=g) < 0.7).to(DEV)[:, :t]
        self.grad_all = torch.full(shape, SENT, dtype=TYPES[kind], device=DEV)
        self.grad = inner(self.grad_all)
        self.loss = torch.full((k,), SENT, device=DEV)
        self.means = torch.full((k, e), SENT, device=DEV)
        self.counts_all = torch.full((k, e + 2), -7, dtype=torch.int64, device=DEV)
        self.counts = self.counts_all[:, 1:1 + e]
        self.totals_all = torch.randint(0, 1 << 40, (k, 2 * e), generator=g).to(DEV)
        self.totals = self.totals_all[:, e:]
        self.scale = (0.5 + torch.rand(k, generator=g, dtype=torch.float64)).to(DEV)
        self.ws = dlc.alloc_expert_balance_workspace(k, t, e, DEV)

    def call(self, **kw):
        args = dict(coef=0.37, mask=self.mask, mean_probs=self.means, grad_logits=self.grad, grad_scale=self.scale,
                    totals=self.totals)
        args.update(kw)
        self.args = args
        self.before = {n: getattr(self, n).clone() for n in ("grad_all", "loss", "means", "counts_all", "totals_all")}
        dlc.dlc_expert_balance(self.x, self.ids, self.loss, self.counts, self.ws, **args)
        torch.cuda.synchronize()

    def check(self, nan_rows=()):
        a, e, t = self.args, self.e, self.t
        want = {n: b.clone() for n, b in self.before.items()}
        for i in range(self.k):
            if a.get("present") is not None and not a["present"][i]:
                continue
            x = widen(self.x[i])
            mask = None if a["mask"] is None else a["mask"][i].cpu().numpy().astype(bool)
            up = 1.0 if a["grad_scale"] is None else float(a["grad_scale"][i])
            loss, counts, means, grad = experts.balance(x, self.ids[i].cpu().numpy(), mask, a["coef"], up)
            kept = np.ones(t, bool) if mask is None else mask
            want["counts_all"][i, 1:1 + e] = torch.from_numpy(counts).to(DEV)
            if a["totals"] is not None:
                want["totals_all"][i, e:] += torch.from_numpy(counts).to(DEV)
            near = x[kept]
            with np.errstate(invalid="ignore"):
                d = near.max(1, keepdims=True) - near if len(near) else np.zeros((1, 1))
            d = d[np.isfinite(d) & (d < 88)]
            r = (4.6 * (float(d.max()) if d.size else 0.0) + 31) * U
            got = float(self.loss[i])
            assert (np.isnan(loss) and np.isnan(got)) or abs(got - loss) <= (r + 17 * U) * abs(loss), (i, got, loss)
            want["loss"][i] = self.loss[i]
            if a["mean_probs"] is not None:
                got = widen(self.means[i])
                assert np.array_equal(np.isnan(got), np.isnan(means))
                assert (np.abs(got - means) <= (r + 17 * U) * means + 2.0 ** -126)[~np.isnan(means)].all()
                want["means"][i] = self.means[i]
            if a["grad_logits"] is not None:
                n = max(1, int(kept.sum()))
                p = np.stack([experts.softmax(row) for row in x]) if t else np.zeros((0, e))
                big = abs(up * a["coef"]) * e / (n * n * self.top) * np.abs(counts - counts.mean()).max()
                first = self.grad.storage_offset() % self.grad.stride(1) if self.grad.stride(1) else 0
                old = widen(self.before["grad_all"][i, :t, first:first + e])
                if a.get("accumulate"):
                    grad = old + grad
                else:
                    p[~kept] = 0
                half = torch.finfo(TYPES[self.kind]).eps / 2
                tol = p * big * (3 * r + 64 * U) * (1 + half) + np.abs(grad) * (half + (U if a.get("accumulate") else 0))
                got = widen(self.grad[i])
                grad[~kept] = old[~kept] if a.get("accumulate") else 0.0
                assert np.array_equal(np.isnan(got), np.isnan(grad))
                ok = np.abs(got - grad) <= tol * (1 + 2.0 ** -10) + TINY[self.kind]
                assert ok[~np.isnan(grad)].all(), (i, np.abs(got - grad)[~ok & ~np.isnan(grad)].max())
                assert (got[~kept] == grad[~kept]).all()
                want["grad_all"][i, :t, first:first + e] = self.grad[i]
        for name, b in want.items():
            got = getattr(self, name)
            assert torch.equal(torch.nan_to_num(got), torch.nan_to_num(b)), name


# --- the balance loss ------------------------------------------------------------------------

@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("e", [1, 2, 3, 7, 8, 9, 15, 16, 17, 31, 33, 60, 64, 65, 100, 128, 200, 255, 256, 257, 300, 511,
                               513, 1000, 1024])
def test_every_width_of_a_router(kind, e):
    r = Router(2, 37, e, min(e, 3), kind, pad=e % 5, first=e % 3, seed=e)
    r.call()
    r.check()


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("e,top,t", [(8, 2, 9001), (60, 4, 5003), (64, 6, 4096), (200, 8, 1111), (256, 8, 2050),
                                     (512, 2, 700), (1024, 64, 333), (5, 5, 20011), (1, 1, 40000), (16, 1, 12345),
                                     (33, 3, 7777), (128, 8, 3000)])
def test_many_tokens_over_many_blocks(kind, e, top, t):
    r = Router(3, t, e, top, kind, ids=torch.int32 if e % 2 else torch.int64, masked=e in (60, 200, 5), pad=e % 4, seed=t)
    r.call(present=[1, 0, 1])
    r.check()
    r.call(grad_logits=None)
    r.check()


@pytest.mark.parametrize("t", [0, 1, 2, 63, 64, 65, 255, 256, 257])
@pytest.mark.parametrize("masked", [False, True])
def test_few_tokens(t, masked):
    r = Router(2, t, 24, 4, "bf16", masked=masked, seed=t)
    r.call()
    r.check()


@pytest.mark.parametrize("t,e", [(40, 12), (3000, 40)])
def test_a_learner_whose_mask_leaves_nothing_has_no_loss(t, e):
    r = Router(3, t, e, 2, "fp32", masked=True)
    r.mask[1] = False
    r.call()
    r.check()
    assert float(r.loss[1]) == 0.0 and not r.counts[1].any() and not r.means[1].any() and not r.grad[1].any()


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("t,e", [(40, 12), (3000, 70)])
def test_what_the_mask_leaves_out_may_hold_anything(kind, t, e):
    r, clean = Router(2, t, e, 2, kind, masked=True, seed=4), Router(2, t, e, 2, kind, masked=True, seed=4)
    clean.x_all[:, :t].masked_fill_(~clean.mask[..., None], 0.25)
    for i, junk in enumerate((float("nan"), float("inf"))):
        r.x[i].masked_fill_(~r.mask[i][:, None], junk)
    r.ids.masked_fill_(~r.mask[..., None], 1 << 30)
    for q in (r, clean):
        q.call()
    for name in ("loss", "means", "counts_all", "totals_all", "grad_all"):
        assert torch.equal(getattr(r, name), getattr(clean, name)), name
    clean.check()


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("factor", [float("inf"), float("nan")])
@pytest.mark.parametrize("t,e", [(40, 12), (3000, 70), (40, 3)])
def test_what_the_mask_leaves_out_has_no_gradient_whatever_the_factor(kind, factor, t, e):
    r = Router(2, t, e, 2, kind, masked=True, seed=4)
    r.mask[1] = False
    r.scale.fill_(factor)
    r.call()
    assert not r.grad[~r.mask].any() and torch.isfinite(r.loss).all()
    assert not torch.isfinite(r.grad[0][r.mask[0]]).all()


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("t,e", [(64, 10), (2500, 48)])
def test_logits_of_impossible_experts(kind, t, e):
    r = Router(1, t, e, 2, kind, seed=8)
    low = torch.finfo(TYPES[kind]).min
    r.x[0, ::3, e // 2:] = float("-inf")
    r.x[0, 1::3, : e // 2] = low
    r.x[0, 5] = float("-inf")   # a token for which nothing is possible
    r.x[0, 6] = low             # the same, written as the lowest value: an even row
    r.call()
    r.check()
    assert not r.grad[0, 5].any()


@pytest.mark.parametrize("value", ["nan", "inf"])
@pytest.mark.parametrize("t,e", [(64, 10), (2500, 48)])
def test_a_logit_that_is_no_number_spoils_its_own_token(value, t, e):
    r = Router(2, t, e, 2, "fp32", seed=9)
    r.x[0, 7, 3] = float(value)
    r.call()
    assert torch.isnan(r.grad[0, 7]).all() and torch.isfinite(r.grad[0, :7]).all() and torch.isfinite(r.grad[0, 8:]).all()
    assert torch.isnan(r.loss[0]) and torch.isfinite(r.loss[1]) and torch.isfinite(r.grad[1]).all()


@pytest.mark.parametrize("ids", [torch.int32, torch.int64])
@pytest.mark.parametrize("t", [50, 4000])
def test_choices_outside_the_experts_are_dropped(ids, t):
    r = Router(2, t, 20, 4, "fp32", ids=ids, seed=3)
    r.ids[:, ::2, 0] = -1
    r.ids[:, 1::3, 1] = 20
    r.ids[:, ::5, 2] = torch.iinfo(ids).max
    r.ids[:, 2::5, 3] = torch.iinfo(ids).min
    if ids is torch.int64:
        r.ids[:, 4::7, 1] = (1 << 32) + 3   # 3 in the low half
    r.ids[:, 3::7, 2] = r.ids[:, 3::7, 0]   # the same expert twice
    r.call()
    r.check()


@pytest.mark.parametrize("t", [33, 6000])
@pytest.mark.parametrize("kind", TYPES)
def test_the_gradient_can_be_added_to(kind, t):
    r = Router(2, t, 36, 3, kind, masked=True, seed=t)
    r.grad.copy_(torch.randn(r.grad.shape, device=DEV) * 1e-3)
    r.call(accumulate=True)
    r.check()


@pytest.mark.parametrize("t", [33, 6000])
def test_layouts_of_the_logits(t):
    """Tokens outermost, one row of logits for all tokens, rows at odd addresses."""
    base = Router(3, t, 30, 3, "bf16", seed=1)
    x = torch.randn((t, 3, 31), device=DEV).bfloat16()
    grad = torch.full((t, 3, 31), SENT, dtype=torch.bfloat16, device=DEV)
    for view, out in ((x.transpose(0, 1)[:, :, 1:], grad.transpose(0, 1)[:, :, 1:]),
                      (x[:1, :, :30].transpose(0, 1).expand(3, t, 30), grad.transpose(0, 1)[:, :, :30])):
        plain = view.contiguous()
        base.x, dense = view, torch.empty_like(plain)
        base.call(grad_logits=out)
        got = [v.clone() for v in (base.loss, base.means, base.counts, out)]
        base.x = plain
        base.call(grad_logits=dense)
        for a, b in zip(got, (base.loss, base.means, base.counts, dense)):
            assert torch.equal(a, b)
    assert (grad[:, :, 0] != SENT).any() and torch.isfinite(grad).all()


@pytest.mark.parametrize("t", [100, 5000])
def test_an_even_router_has_the_least_loss_and_no_gradient(t):
    e = 8
    r = Router(1, t * e, e, 1, "fp32")
    r.x.zero_()
    r.ids[0, :, 0] = torch.arange(t * e, device=DEV) % e
    r.call()
    assert float(r.loss) == pytest.approx(0.37, rel=2e-7) and not r.grad.any()
    r.x[0, :, 2] = 100.0
    r.ids.fill_(2)
    r.call()
    assert float(r.loss) == pytest.approx(0.37 * e, rel=2e-7)


def test_the_gradient_is_the_losss():
    """Central differences of the GPU's own loss, in the direction of the gradient and in others."""
    r = Router(1, 48, 12, 2, "fp32", seed=5, skew=2.0)
    r.call(grad_scale=None)
    x, g = r.x.clone(), r.grad.double().clone()
    gen = torch.Generator(DEV).manual_seed(1)
    for way in (g / g.norm(), torch.randn(x.shape, device=DEV, generator=gen).double()):
        h = 0.5 / float(way.abs().max())
        f = []
        for sign in (1, -1):
            r.x.copy_(x + sign * h * way)
            loss, *_ = experts.balance(widen(r.x[0]), r.ids[0].cpu().numpy(), None, 0.37)
            r.call(grad_scale=None)
            assert abs(float(r.loss) - loss) <= 200 * U * loss
            f.append(float(r.loss))
        slope = (f[0] - f[1]) / (2 * h)
        # the third derivative of a mean of softmaxes along `way` is at most the loss times (2 max|way|)^3
        bound = 0.37 * 12 * (2 * float(way.abs().max())) ** 3 * h * h / 6 + 300 * U * f[0] / h
        assert abs(slope - float((g * way).sum())) <= bound


def test_a_masked_batch_gives_what_its_kept_tokens_give():
    r = Router(1, 3001, 50, 3, "fp32", masked=True, seed=6)
    r.call()
    keep = torch.nonzero(r.mask[0])[:, 0]
    q = Router(1, len(keep), 50, 3, "fp32", seed=6)
    q.x.copy_(r.x[:, keep])
    q.ids.copy_(r.ids[:, keep])
    q.scale.copy_(r.scale)
    q.call()
    assert torch.equal(q.counts, r.counts)
    assert torch.equal(q.grad, r.grad[:, keep])   # a token's gradient depends on the counts alone
    assert abs(float(q.loss) - float(r.loss)) <= 34 * U * float(q.loss)


def test_repeated_calls_agree_and_totals_grow():
    r = Router(4, 9000, 96, 4, "bf16", seed=2)
    r.call()
    first = [v.clone() for v in (r.loss, r.means, r.counts, r.grad)]
    start = r.before["totals_all"].clone()
    for _ in range(3):
        r.call()
        for a, b in zip(first, (r.loss, r.means, r.counts, r.grad)):
            assert torch.equal(a, b)
    assert torch.equal(r.totals, start[:, r.e:] + 4 * r.counts)


# --- the merge ---------------------------------------------------------------------------------

class Outer:
    """Codes, codebooks and state of an outer step with values in everything that is not the call's."""

    def __init__(self, sizes, k, experts_of=None, seed=0, weights=None, absent=()):
        g = torch.Generator().manual_seed(seed)
        at, self.tensors = 64, []
        for j, n in enumerate(sizes):
            self.tensors.append((at + 64, at, n))
            at += -(-n // 64) * 64 + (64 if j % 3 == 0 else 0)
        self.k, self.stride, nt = k, at + 64, len(sizes)
        self.codes = torch.randint(0, 256, (k, self.stride), generator=g, dtype=torch.uint8).to(DEV)
        self.codebook = torch.randn((k, nt, 256), generator=g).to(DEV)
        self.theta = torch.randn(self.stride + 64, generator=g).to(DEV)
        self.mom = torch.randn(self.stride + 64, generator=g).to(DEV)
        self.weights = weights or [float(x) for x in torch.rand(k, generator=g) + 0.1]
        for i in absent:
            self.weights[i] = 0.0
            self.codebook[i] = float("nan")
        self.expert_of = experts_of or [j % 4 - 1 for j in range(nt)]
        self.counts = torch.randint(0, 1 << 20, (k, 5), generator=g).to(DEV)
        self.share = torch.full((nt, k), SENT, dtype=torch.float64, device=DEV)
        self.norm, self.scale = (torch.full((1,), SENT, dtype=torch.float64, device=DEV) for _ in range(2))
        self.ws = dlc.alloc_outer_grad_norm_workspace(self.tensors, DEV)

    def shares(self, **kw):
        dlc.dlc_expert_weights(self.counts, self.weights, self.expert_of, self.share, **kw)
        want = experts.tensor_weights(self.counts.cpu().numpy(), self.weights, self.expert_of, kw.get("token_weight"))
        assert np.array_equal(self.share.cpu().numpy(), want)
        return want

    def check_norm(self, share, max_norm=float("inf")):
        dlc.dlc_outer_grad_norm(self.codes, self.codebook, self.weights, self.tensors, self.norm, self.scale, self.ws,
                                max_norm=max_norm, tensor_weights=None if share is None else self.share)
        norm, scale = experts.outer_grad_norm(self.codes.cpu().numpy(), self.codebook.cpu().numpy(), self.weights,
                                              self.tensors, share, max_norm)
        assert abs(float(self.norm) - norm) <= 2.0 ** -40 * norm and abs(float(self.scale) - scale) <= 2.0 ** -40 * scale
        return float(self.scale)

    def check_step(self, share, scale):
        th, mo = self.theta.cpu().numpy().copy(), self.mom.cpu().numpy().copy()
        factor = None if scale is None else torch.tensor([scale], dtype=torch.float64, device=DEV)
        dlc.dlc_merge_clipped_step(self.theta, self.mom, self.codes, self.codebook, self.weights, self.tensors,
                                   grad_scale=factor, tensor_weights=None if share is None else self.share)
        experts.clipped_step(th, mo, self.codes.cpu().numpy(), self.codebook.cpu().numpy(), self.weights, self.tensors,
                             share, scale)
        assert np.array_equal(self.theta.cpu().numpy(), th) and np.array_equal(self.mom.cpu().numpy(), mo)


LISTS = {"large": [1 << 21, 3, 500_001, 70_000], "one": [1], "vectors": [4096] * 4, "edges": [63, 64, 65, 4095, 4096, 4097, 8191, 8193, 1, 2],
         "ragged": [1, 100003, 65, 64 * 300 + 9, 31, 77777], "many": [(37 * i) % 700 + 1 for i in range(400)]}


@pytest.mark.parametrize("name", LISTS)
@pytest.mark.parametrize("k", [1, 2, 3, 8, 14, 25])
def test_norm_and_step(name, k):
    o = Outer(LISTS[name], k, seed=k, absent=(1,) if k > 2 else ())
    o.check_norm(None)
    o.check_step(None, None)
    share = o.shares()
    scale = o.check_norm(share, max_norm=0.5)
    o.check_step(share, scale)
    o.check_step(share, 0.125)


def test_sixty_four_learners():
    o = Outer([5000, 1, 777], 64, seed=3, absent=(0, 63))
    share = o.shares(token_weight=[0.5 + i / 64 for i in range(64)])
    o.check_step(share, o.check_norm(share, 1.0))


@pytest.mark.parametrize("bad", [0.0, -1.0, float("nan"), float("inf")])
def test_a_factor_that_is_no_factor_leaves_the_step_out(bad):
    o = Outer(LISTS["ragged"], 3)
    o.check_step(None, bad)


def test_without_weights_and_factor_it_is_the_outer_step():
    o = Outer(LISTS["ragged"], 5, seed=1, absent=(2,))
    th, mo = o.theta.clone(), o.mom.clone()
    dlc.dlc_merge_outer_step(th, mo, o.codes, o.codebook, o.weights, o.tensors)
    dlc.dlc_merge_clipped_step(o.theta, o.mom, o.codes, o.codebook, o.weights, o.tensors)
    assert torch.equal(th, o.theta) and torch.equal(mo, o.mom)


@pytest.mark.parametrize("sizes", [LISTS["edges"], LISTS["ragged"], LISTS["large"]])
def test_a_gradient_that_is_not_finite_is_left_out(sizes):
    o = Outer(sizes, 2)
    o.codebook[1, 3, :] = float("inf")
    dlc.dlc_outer_grad_norm(o.codes, o.codebook, o.weights, o.tensors, o.norm, o.scale, o.ws, max_norm=1.0)
    assert not torch.isfinite(o.norm) and float(o.scale) == 0.0
    th, mo = o.theta.clone(), o.mom.clone()
    dlc.dlc_merge_clipped_step(o.theta, o.mom, o.codes, o.codebook, o.weights, o.tensors, grad_scale=o.scale)
    assert torch.equal(th, o.theta) and torch.equal(mo, o.mom)


@pytest.mark.parametrize("n", [1, 4095, 5000, 100_001, 2_300_001])
@pytest.mark.parametrize("k", [2, 6])
def test_entries_that_no_code_of_the_tensor_names_do_not_count(n, k):
    """Codes behind a tensor's end, in its last group of 64, name entries that may hold anything."""
    o = Outer([n, 70], k, seed=n)
    used = torch.zeros(o.stride, dtype=torch.bool, device=DEV)
    for _, at, m in o.tensors:
        used[at:at + m] = True
    o.codes[:, used] = o.codes[:, used].clamp(max=253)
    o.codes[:, ~used] = 254
    o.codes[0, ~used] = 255
    o.codebook[..., 254] = float("inf")
    o.codebook[..., 255] = float("nan")
    o.check_step(None, o.check_norm(None, 0.5))


def test_a_gradient_of_zero_has_norm_zero_and_is_not_clipped():
    o = Outer([100, 5000], 2)
    o.codebook.zero_()
    dlc.dlc_outer_grad_norm(o.codes, o.codebook, o.weights, o.tensors, o.norm, o.scale, o.ws, max_norm=1.0)
    assert float(o.norm) == 0.0 and float(o.scale) == 1.0
    o = Outer([100, 5000, 2_170_000], 2)
    o.codebook.zero_()
    dlc.dlc_outer_grad_norm(o.codes, o.codebook, o.weights, o.tensors, o.norm, o.scale, o.ws, max_norm=1.0)
    assert float(o.norm) == 0.0 and float(o.scale) == 1.0


@pytest.mark.parametrize("sizes", [[2000], [100000, 3, 4097], [2_200_000, 3, 4097]])
@pytest.mark.parametrize("size", [1e-44, 1e-20, 1e20, 3e38])
def test_codebooks_of_every_size(sizes, size):
    """From subnormal entries to the largest, one tensor's far from another's."""
    o = Outer(sizes, 3, seed=4)
    o.codebook.mul_(size / float(o.codebook.abs().max()))
    o.codebook[:, -1] *= 0.125
    o.check_norm(None, size)


@pytest.mark.parametrize("n", [70000, 2_300_000])
def test_learners_that_nearly_cancel(n):
    o = Outer([n], 2, weights=[1.0, 1.0])
    o.codes[1].copy_(o.codes[0])
    o.codebook[1].copy_(-o.codebook[0])
    o.codebook[1, 0, 7] *= 1 + 2.0 ** -20
    o.check_norm(None)


def test_experts_that_nobody_used_and_learners_that_did_not():
    o = Outer([70, 80, 90, 100, 110], 3, experts_of=[0, 1, 2, -1, 4])
    o.counts[:, 0] = 0
    o.counts[:, 1] = torch.tensor([0, 5, 0])
    o.counts[:, 2] = torch.tensor([-3, 1, 1])
    o.codebook[0, 1] = float("nan")   # has no part in its expert's tensor
    o.codebook[2, 1] = float("inf")
    share = o.shares()
    assert share[1].tolist() == [0.0, 1.0, 0.0] and share[2].tolist() == [0.0, 0.5, 0.5]
    o.check_step(share, o.check_norm(share, 2.0))


def test_a_thousand_tensors_of_experts():
    o = Outer([65] * 1500, 4, seed=2, experts_of=[j % 6 - 1 for j in range(1500)], absent=(3,))
    share = o.shares(token_weight=[1.0, 0.25, 0.0, 1.0])
    o.check_step(share, o.check_norm(share, 3.0))


# --- together -----------------------------------------------------------------------------------

def test_learners_route_count_and_merge():
    """Two layers of four experts on three learners: inner steps count, the outer step weighs, clips and merges;
    eagerly and replayed from one graph, on streams of their own, with eager work between."""
    k, e, layers, steps = 3, 4, 2, 3
    o = Outer([640, 1000, 1000, 1000, 1000, 63, 999, 999, 999, 999], k, seed=4,
              experts_of=[-1, 0, 1, 2, 3, -1, 4, 5, 6, 7])
    totals = torch.zeros((k, layers * e), dtype=torch.int64, device=DEV)
    routers = [Router(k, 200 if s else 5000, e, 2, "bf16", seed=s) for s in range(layers * steps)]
    clip = torch.zeros(1, dtype=torch.float64, device=DEV)

    def go():
        totals.zero_()
        for s, r in enumerate(routers):
            layer = s % layers
            dlc.dlc_expert_balance(r.x, r.ids, r.loss, r.counts, r.ws, coef=0.01, grad_logits=r.grad,
                                   totals=totals[:, layer * e:(layer + 1) * e])
        dlc.dlc_expert_weights(totals, o.weights, o.expert_of, o.share)
        dlc.dlc_outer_grad_norm(o.codes, o.codebook, o.weights, o.tensors, o.norm, clip, o.ws, max_norm=5.0,
                                tensor_weights=o.share)
        dlc.dlc_merge_clipped_step(o.theta, o.mom, o.codes, o.codebook, o.weights, o.tensors, grad_scale=clip,
                                   tensor_weights=o.share)

    th0, mo0 = o.theta.clone(), o.mom.clone()
    go()
    torch.cuda.synchronize()
    want = [v.clone() for v in (totals, o.share, o.norm, clip, o.theta, o.mom, *(r.grad for r in routers))]
    counted = sum(experts.balance(widen(r.x[0]), r.ids[0].cpu().numpy())[1] for r in routers[::2])
    assert totals[0, :e].tolist() == counted.tolist()
    share = experts.tensor_weights(totals.cpu().numpy(), o.weights, o.expert_of)
    assert np.array_equal(o.share.cpu().numpy(), share) and 0.0 < float(clip) < 1.0
    th, mo = th0.cpu().numpy().copy(), mo0.cpu().numpy().copy()
    experts.clipped_step(th, mo, o.codes.cpu().numpy(), o.codebook.cpu().numpy(), o.weights, o.tensors, share, float(clip))
    assert np.array_equal(th, o.theta.cpu().numpy()) and np.array_equal(mo, o.mom.cpu().numpy())

    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            go()
    torch.cuda.current_stream().wait_stream(side)
    for _ in range(4):
        o.theta.copy_(th0)
        o.mom.copy_(mo0)
        o.ws.fill_(255)
        for r in routers:
            r.ws.fill_(255)
            r.grad.zero_()
        noise = torch.randn(1 << 18, device=DEV).sum()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.isfinite(noise)
        for a, b in zip(want, (totals, o.share, o.norm, clip, o.theta, o.mom, *(r.grad for r in routers))):
            assert torch.equal(a, b)


def test_two_streams_at_once():
    routers = [Router(2, 20000, 64, 4, "bf16", seed=s) for s in range(2)]
    for r in routers:
        r.call()
    want = [(r.loss.clone(), r.grad.clone(), r.counts.clone()) for r in routers]
    streams = [torch.cuda.Stream() for _ in routers]
    torch.cuda.synchronize()
    for _ in range(5):
        for r, s in zip(routers, streams):
            dlc.dlc_expert_balance(r.x, r.ids, r.loss, r.counts, r.ws, coef=0.37, grad_logits=r.grad,
                                   grad_scale=r.scale, stream=s)
    torch.cuda.synchronize()
    for r, w in zip(routers, want):
        assert all(torch.equal(a, b) for a, b in zip((r.loss, r.grad, r.counts), w))


def test_rows_further_apart_than_32_bits_count():
    """Tokens 2^26 elements apart, and a tensor past 2^32 bytes of a row of codes."""
    t, e, far = 66, 16, 1 << 26
    near = Router(1, t, e, 2, "bf16", masked=True, seed=11)
    buf = torch.zeros(t * far, dtype=torch.bfloat16, device=DEV)
    q = Router(1, t, e, 2, "bf16", masked=True, seed=11)
    q.x = buf.as_strided((1, t, e), (0, far, 1))
    q.x.copy_(near.x)
    out = buf.as_strided((1, t, e), (0, far, 1), storage_offset=64)
    spare = torch.zeros((1, t, e), dtype=torch.bfloat16, device=DEV)
    near.call(grad_logits=spare)
    with pytest.raises(dlc.DlcError, match="overlap"):  # its rows lie between the logits' rows
        q.call(grad_logits=out)
    del out
    q.call(grad_logits=None)
    assert torch.equal(q.loss, near.loss) and torch.equal(q.counts, near.counts)
    logits = near.x
    q.x = logits
    out = buf.as_strided((1, t, e), (0, far, 1))
    q.call(grad_logits=out)
    assert torch.equal(out, spare) and torch.equal(q.loss, near.loss)
    del buf, out, q
    stride, n = (1 << 32) + 128 * 64, 5001
    g = torch.Generator().manual_seed(0)
    codes = torch.zeros((2, stride), dtype=torch.uint8, device=DEV)
    lo = stride - 5056
    codes[:, lo:] = torch.randint(0, 256, (2, 5056), generator=g, dtype=torch.uint8).to(DEV)
    o = Outer([n], 2, seed=1)
    far_tensors = [(o.tensors[0][0], lo, n)]
    _, at, _ = o.tensors[0]
    o.codes[:, at:at + 5056] = codes[:, lo:]
    dlc.dlc_outer_grad_norm(o.codes, o.codebook, o.weights, o.tensors, o.norm, o.scale, o.ws, max_norm=1.0)
    norm, scale = torch.zeros_like(o.norm), torch.zeros_like(o.scale)
    dlc.dlc_outer_grad_norm(codes, o.codebook, o.weights, far_tensors, norm, scale, o.ws, max_norm=1.0)
    assert torch.equal(norm, o.norm) and torch.equal(scale, o.scale) and float(norm) > 0
    th, mo = o.theta.clone(), o.mom.clone()
    dlc.dlc_merge_clipped_step(o.theta, o.mom, o.codes, o.codebook, o.weights, o.tensors, grad_scale=scale)
    dlc.dlc_merge_clipped_step(th, mo, codes, o.codebook, o.weights, far_tensors, grad_scale=scale)
    assert torch.equal(th, o.theta) and torch.equal(mo, o.mom)


def test_one_workspace_serves_calls_in_a_row():
    """Of several sizes and kinds on one stream, without waiting in between."""
    routers = [Router(2, t, e, 2, kind, seed=t, masked=t % 2 == 0)
               for t, e, kind in ((6000, 48, "bf16"), (37, 300, "fp32"), (2500, 128, "fp16"), (9000, 8, "bf16"))]
    ws = max((r.ws for r in routers), key=lambda w: w.numel())
    for r in routers:
        r.ws = ws
    torch.cuda.synchronize()
    for grad in (True, False):
        for r in routers:
            r.args = dict(coef=0.37, mask=r.mask, mean_probs=r.means, grad_scale=r.scale, totals=r.totals,
                          grad_logits=r.grad if grad else None)
            r.before = {n: getattr(r, n).clone() for n in ("grad_all", "loss", "means", "counts_all", "totals_all")}
            dlc.dlc_expert_balance(r.x, r.ids, r.loss, r.counts, r.ws, **r.args)
        for r in routers:
            r.check()
