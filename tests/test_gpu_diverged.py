"""A learner that diverged shows in the outer step: NaN and infinite parameters are outside the contract of the
quantizing calls, which stay within their buffers, but without DLC_DEBUG_CHECKS the step's own result is the only
sign of them.  It is left in the tensors that hold them and in no other."""
import pytest
import torch

import diloco_outer_step_amd as dlc
from tests.test_gpu_rda import packed, rda_buffers

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.mark.parametrize("junk", [float("nan"), float("inf")])
@pytest.mark.parametrize("k,bad", [(1, [0]), (3, [0, 1, 2]), (3, [1]), (5, [4])])
def test_a_diverged_learner_shows_in_the_step_merged_by_averaged_directions(junk, k, bad):
    tensors, stride = packed([5000, 70, 3 * 4096 + 5, 64])
    g = torch.Generator().manual_seed(k)
    theta_g = (torch.randn(stride, generator=g) * 0.02).to(DEV)
    theta_L = (theta_g + torch.randn((k, stride), generator=g).to(DEV) * 1e-3).contiguous()
    momentum = (torch.randn(stride, generator=g) * 1e-3).to(DEV)
    weights = [1.0 + i for i in range(k)]
    out = []
    for spoil in (False, True):
        for t in (1, 2) if spoil else ():
            _, lo, n = tensors[t]
            theta_L[bad, lo:lo + n] = junk
        codes, cb, rng, norms, ws = rda_buffers(k, stride, len(tensors), tensors)
        th, mo = theta_g.clone(), momentum.clone()
        dlc.dlc_rda_outer_step(th, mo, theta_L, tensors, weights, codes, cb, rng, norms, ws, 0.7, 0.9)
        torch.cuda.synchronize()
        out.append((th, mo))
    (th, mo), (th_bad, mo_bad) = out
    for t, (off, _, n) in enumerate(tensors):
        a, b = th_bad[off:off + n], mo_bad[off:off + n]
        if t in (1, 2):
            assert torch.isnan(a).any() and torch.isnan(b).any(), t
        else:
            assert torch.equal(a, th[off:off + n]) and torch.equal(b, mo[off:off + n]), t
