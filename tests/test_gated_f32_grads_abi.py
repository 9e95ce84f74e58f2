"""The gated product's backward call with fp32 gradients of the weights, without a GPU:
arguments are refused with the documented codes before anything is launched."""
import ctypes

import pytest

from level_haar_wavelet_amd import _native

OK, NULL, SHAPE, UNSUPPORTED, WORKSPACE, HIP, ALIAS = range(7)
BIG = 1 << 50
NAMES = ("x", "dh", "wg", "wu", "bg", "bu", "dx", "dwg", "dwu", "dbg", "dbu", "ws")


def at(i):
    return 0x10000000 * (i + 1)


@pytest.mark.parametrize("dtype", range(3))
def test_arguments_are_refused(dtype):
    lib = _native.load()
    d = _native.GatedDesc(100, 64, 96, dtype, 2)
    out = ctypes.c_size_t(0)
    assert lib.wtconv_gated_workspace_size(ctypes.byref(d), 3, ctypes.byref(out)) == OK
    need = out.value

    def bwd(nbytes=need, desc=d, **kw):
        args = [kw.get(n, at(i)) for i, n in enumerate(NAMES)]
        return lib.wtconv_gated_backward_f32_grads(ctypes.byref(desc), *args, nbytes, None)

    for bad, expect in ((_native.GatedDesc(0, 64, 96, dtype, 2), SHAPE), (_native.GatedDesc(100, 64, 96, 3, 2), UNSUPPORTED),
                        (_native.GatedDesc(100, 64, 96, dtype, 4), UNSUPPORTED)):
        assert bwd(desc=bad) == expect
    for k in ("x", "dh", "wg", "wu", "dwg", "dwu", "dbg", "dbu"):
        assert bwd(**{k: None}) == NULL
    assert bwd(dx=None, dwg=None, dwu=None, dbg=None, dbu=None) == NULL
    # fp32 gradients: on 4 bytes, whatever the activations' type
    for k in ("dwg", "dwu"):
        assert bwd(**{k: at(20) + 2}) == UNSUPPORTED
    assert bwd(ws=None) == WORKSPACE and bwd(nbytes=need - 1) == WORKSPACE and bwd(ws=at(11) + 16) == UNSUPPORTED
    # ... and of 4 bytes an element
    last = 96 * 64 * 4 - 4
    assert bwd(dwu=at(7) + last) == ALIAS and bwd(dbg=at(8) + last) == ALIAS and bwd(dx=at(7) + last) == ALIAS
    assert bwd(dwg=at(2) + 4) == ALIAS and bwd(ws=at(7)) == ALIAS
