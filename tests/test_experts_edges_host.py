"""More refusals of the mixture-of-experts calls, on host tensors and made-up addresses: nothing is launched."""
import pytest
import torch

import diloco_outer_step_amd as dlc


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
