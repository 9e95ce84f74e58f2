"""The gated product on the GPU with x and the weights at any element's address."""
import pytest
import torch

import level_haar_wavelet_amd as wt
from tests.block_util import DTYPES, Gated64, check
from tests.test_gpu_gated import NAMES, make

pytestmark = pytest.mark.gpu
CODES = {"f32": 0, "f16": 1, "bf16": 2}


# few rows, short rows and long ones; 16-bit rows of which 8 divides the one, and is copied
@pytest.mark.parametrize("m,c,f", [(3, 64, 40), (40, 61, 43), (64, 1000, 24), (150, 64, 40), (150, 61, 43),
                                   (300, 260, 132), (129, 33, 65)])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("offset", [1, 2, 3])
def test_results(m, c, f, dtype, offset):
    x, wg, wu, bg, bu, dh = make(m, c, f, dtype, seed=m + offset, offset=offset)
    assert x.data_ptr() % 16 and wg.data_ptr() % 16
    ref = Gated64(x, wg, wu, bg, bu, "silu")
    h = wt.wtconv_gated_forward(x, wg, wu, bg, bu)
    check("h", h, ref.h, ref.h_tol())
    want = ref.backward(dh)
    for name, got in zip(NAMES, wt.wtconv_gated_backward(x, dh, wg, wu, bg, bu)):
        check(name, got, *want[name])


@pytest.mark.parametrize("m", [64, 4000])
@pytest.mark.parametrize("dtype,c", [("f32", 256), ("f32", 100), ("bf16", 252), ("f16", 61)])
def test_nothing_is_copied(dtype, c, m):
    """Calls that can take the addresses as they are allocate nothing beside what they are given."""
    f = 64
    x, wg, wu, bg, bu, dh = make(m, c, f, dtype, offset=1)
    work = [torch.empty(wt.wtconv_gated_workspace_size(x.shape, f, CODES[dtype], op), dtype=torch.uint8, device="cuda")
            for op in (0, 3)]
    h = torch.empty_like(dh)
    outs = dict(dx=torch.empty_like(x), dw_gate=torch.empty_like(wg), dw_up=torch.empty_like(wu),
                db_gate=torch.empty_like(bg), db_up=torch.empty_like(bu))
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    wt.wtconv_gated_forward(x, wg, wu, bg, bu, h=h, workspace=work[0])
    wt.wtconv_gated_backward(x, dh, wg, wu, bg, bu, workspace=work[1], **outs)
    torch.cuda.synchronize()
    assert torch.cuda.max_memory_allocated() == before
