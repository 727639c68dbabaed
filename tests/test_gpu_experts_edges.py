"""The mixture-of-experts calls on the GPU, in the corners that tests/test_gpu_experts.py leaves: same oracle, same
tolerances."""
import pytest
import torch

import diloco_outer_step_amd as dlc
from tests.test_gpu_experts import DEV, LISTS, TYPES, Outer, Router

pytestmark = pytest.mark.gpu


# --- merge weights that are a view ----------------------------------------------------------------

def views_of(share):
    """The same [T, K] weights in layouts that are not contiguous."""
    wide = torch.full((share.shape[0], 2 * share.shape[1] + 1), float("nan"), dtype=torch.float64, device=DEV)
    wide[:, 1::2] = share
    return {"learner-major": share.T.contiguous().T, "every other column": wide[:, 1::2]}


@pytest.mark.parametrize("name", ["edges", "ragged", "many"])
@pytest.mark.parametrize("k", [2, 5])
def test_merge_weights_may_be_any_view(name, k):
    o = Outer(LISTS[name], k, seed=k)
    o.shares()
    args = (o.codes, o.codebook, o.weights, o.tensors)
    dlc.dlc_outer_grad_norm(*args, o.norm, o.scale, o.ws, max_norm=0.5, tensor_weights=o.share)
    th, mo = o.theta.clone(), o.mom.clone()
    dlc.dlc_merge_clipped_step(th, mo, *args, grad_scale=o.scale, tensor_weights=o.share)
    side = torch.cuda.Stream()
    for view in views_of(o.share).values():
        assert not view.is_contiguous()
        for stream in (None, side, side.cuda_stream, 0):
            norm, scale = torch.zeros_like(o.norm), torch.zeros_like(o.scale)
            a, b = o.theta.clone(), o.mom.clone()
            torch.cuda.synchronize()
            dlc.dlc_outer_grad_norm(*args, norm, scale, o.ws, max_norm=0.5, tensor_weights=view, stream=stream)
            dlc.dlc_merge_clipped_step(a, b, *args, grad_scale=scale, tensor_weights=view, stream=stream)
            torch.cuda.synchronize()
            assert torch.equal(norm, o.norm) and torch.equal(scale, o.scale)
            assert torch.equal(a, th) and torch.equal(b, mo)


def test_merge_weights_that_are_one_row_for_all_tensors():
    o = Outer(LISTS["edges"], 3, seed=2)
    row = torch.tensor(o.weights, dtype=torch.float64, device=DEV)
    row /= row.sum()
    o.share.copy_(row.expand_as(o.share))
    norms = []
    for share in (o.share, row.expand_as(o.share)):
        dlc.dlc_outer_grad_norm(o.codes, o.codebook, o.weights, o.tensors, o.norm, o.scale, o.ws, tensor_weights=share)
        norms.append(o.norm.clone())
    assert torch.equal(*norms) and float(norms[0]) > 0


def test_a_view_of_merge_weights_in_a_graph():
    """Every replay reads the weights that stand in the view then."""
    o = Outer(LISTS["ragged"], 4, seed=6)
    o.shares()
    first = o.share.clone()
    view = views_of(first)["learner-major"]
    args = (o.codes, o.codebook, o.weights, o.tensors)
    th0, mo0 = o.theta.clone(), o.mom.clone()

    def go():
        dlc.dlc_outer_grad_norm(*args, o.norm, o.scale, o.ws, max_norm=0.5, tensor_weights=view)
        dlc.dlc_merge_clipped_step(o.theta, o.mom, *args, grad_scale=o.scale, tensor_weights=view)

    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        go()
        side.synchronize()
        with torch.cuda.graph(graph, stream=side):
            go()
    for factor in (1.0, 0.5, 2.0):
        view.copy_(first * factor)
        o.theta.copy_(th0)
        o.mom.copy_(mo0)
        go()
        torch.cuda.synchronize()
        want = [v.clone() for v in (o.norm, o.scale, o.theta, o.mom)]
        o.theta.copy_(th0)
        o.mom.copy_(mo0)
        o.norm.zero_()
        o.scale.zero_()
        noise = torch.randn(1 << 18, device=DEV).mul(3.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.isfinite(noise).all()
        assert all(torch.equal(x, y) for x, y in zip(want, (o.norm, o.scale, o.theta, o.mom)))


# --- tokens for which nothing is possible ----------------------------------------------------------

@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("factor", [float("inf"), float("nan"), -float("inf"), 1.5])
@pytest.mark.parametrize("t,e,masked", [(40, 12, False), (41, 3, True), (3000, 70, True), (2501, 300, False), (600, 1000, True)])
def test_a_token_of_no_possible_expert_has_no_gradient_whatever_the_factor(kind, factor, t, e, masked):
    """One that the mask keeps, and whose logits are all -infinity: the overflowed loss scale of a step that will be
    left out must not spoil a gradient that is added to."""
    for accumulate in (False, True):
        r = Router(2, t, e, 2, kind, masked=masked, seed=t)
        none = torch.zeros((2, t), dtype=torch.bool, device=DEV)
        none[:, ::7] = True
        none[1, t // 2:] = True
        r.x.masked_fill_(none[..., None], float("-inf"))
        r.scale[0] = factor
        if accumulate:
            r.grad.copy_(torch.randn(r.grad.shape, device=DEV))
        before = r.grad.clone()
        r.call(accumulate=accumulate)
        left = none if r.mask is None else none | ~r.mask
        want = before if accumulate else torch.zeros_like(before)
        assert torch.equal(r.grad[left], want[left])
        assert torch.isfinite(r.loss).all() and torch.isfinite(r.means).all() and torch.isfinite(r.grad[1]).all()
        assert bool(torch.isfinite(r.grad[0][~left[0]]).all()) == (factor == 1.5)
        if factor == 1.5:
            r.check()


def test_the_workspace_of_the_longest_batch_serves_a_shorter_one():
    r = Router(2, 3927, 512, 8, "bf16", seed=3)
    r.ws = dlc.alloc_expert_balance_workspace(2, 4551, 512, DEV)
    guard = torch.full((r.ws.numel() + 512,), 255, dtype=torch.uint8, device=DEV)
    start = -guard.data_ptr() % 256
    r.ws = guard[start:start + r.ws.numel()]
    for grad in (None, r.grad):
        r.call(grad_logits=grad)
        r.check()
    assert (guard[start + r.ws.numel():] == 255).all()


# --- the norm's rounds of learners -----------------------------------------------------------------

@pytest.mark.parametrize("name", ["large", "ragged", "edges", "many"])
@pytest.mark.parametrize("k,absent", [(4, ()), (5, ()), (5, (0,)), (8, ()), (9, (3,)), (12, ()), (16, ()), (17, ())])
def test_norm_and_step_of_whole_and_broken_rounds_of_learners(name, k, absent):
    """Four learners are an instantiation of their own, more take rounds of four; up to sixteen fit the one block."""
    o = Outer(LISTS[name], k, seed=k, absent=absent)
    o.check_norm(None)
    share = o.shares()
    o.check_step(share, o.check_norm(share, max_norm=0.5))


@pytest.mark.parametrize("k", [1, 4, 16])
def test_the_norm_of_a_few_tiles_with_any_number_of_learners(k):
    o = Outer(LISTS["vectors"], k, seed=k)
    share = o.shares()
    o.check_step(share, o.check_norm(share, max_norm=0.5))
