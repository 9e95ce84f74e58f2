"""Which device the gradient norm and clipping take, on the GPU."""
import pytest
import torch

import level_haar_wavelet_amd as wt
from level_haar_wavelet_amd.optim import clip_grad_norm_

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("device", ["cuda", torch.device("cuda"), "cuda:0", 0], ids=str)
def test_device_without_an_index(device):
    """A device without an index is the one that the gradients lie on, or else the current one."""
    g = torch.full((9,), 2.0, device="cuda:0")
    norm = wt.wtconv_grad_norm([g], device=device)
    assert norm.device == g.device and float(norm) == 6.0
    norm, out = wt.wtconv_clip_grad_norm([g], 3.0, eps=0.0, device=device)
    assert float(norm) == 6.0 and out[0] is g and bool((g == 1.0).all())
    empty = wt.wtconv_grad_norm([], device=device)
    assert empty.device == torch.device("cuda", torch.cuda.current_device()) and float(empty) == 0


def test_another_device_is_refused():
    g = torch.ones(3, device="cuda")
    for device in ("cpu", "cuda:1"):
        with pytest.raises(TypeError, match="lies on"):
            wt.wtconv_grad_norm([g], device=device)


def test_parameters_without_gradients_lie_anywhere():
    p = [torch.nn.Parameter(torch.ones(4, device=d)) for d in ("cpu", "meta", "cuda", "cuda")]
    p[2].grad, p[3].grad = torch.full((4,), 3.0, device="cuda"), torch.full((4,), 4.0, device="cuda")
    assert float(clip_grad_norm_(p, 5.0, eps=0.0)) == 10.0
    assert bool((p[2].grad == 1.5).all()) and bool((p[3].grad == 2.0).all()) and p[0].grad is None
    with pytest.raises(TypeError, match="GPU"):
        clip_grad_norm_(p[:2], 1.0)
    # none has a gradient: the norm comes on the GPU that one of them lies on
    norm = clip_grad_norm_([p[0], torch.nn.Parameter(torch.ones(2, device="cuda"))], 1.0)
    assert norm.device == p[2].device and float(norm) == 0
