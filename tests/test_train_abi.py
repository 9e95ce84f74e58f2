"""Group norm, Newton-Schulz and Muon entry points without a GPU: descriptors and
arguments are refused with the documented codes before anything is launched,
and the binding refuses tensors that the entry points cannot take."""
import ctypes
import os
import subprocess
import sys

import pytest
import torch

import level_haar_wavelet_amd as wt
from level_haar_wavelet_amd import _native

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, NULL, SHAPE, UNSUPPORTED, WORKSPACE, HIP, ALIAS = range(7)


@pytest.fixture(scope="module")
def lib():
    return _native.load()


def norm_desc(n=2, c=8, h=4, w=4, groups=2, dtype=0, act=0, xl=0, yl=0, eps=1e-5):
    return _native.NormDesc(n, c, h, w, groups, dtype, act, xl, yl, eps)


def ortho_desc(batch=1, rows=80, cols=120, dtype=0, steps=5, eps=1e-7):
    return _native.OrthoDesc(batch, rows, cols, dtype, steps, eps)


BAD_NORM = [
    (dict(n=0), SHAPE), (dict(c=0), SHAPE), (dict(h=0), SHAPE), (dict(w=-1), SHAPE), (dict(groups=0), SHAPE),
    (dict(groups=3), SHAPE), (dict(groups=16), SHAPE), (dict(h=1 << 20, w=1 << 20), SHAPE),
    (dict(c=1 << 16, h=1 << 8, w=1 << 8, groups=1), SHAPE),
    (dict(c=1, h=1, w=(1 << 31) - 1, groups=1), SHAPE), (dict(n=1 << 62, c=2), SHAPE), (dict(n=1 << 20, c=8), SHAPE),
    (dict(n=1 << 62), SHAPE), (dict(h=1 << 62), SHAPE), (dict(eps=0.0), SHAPE), (dict(eps=-1.0), SHAPE),
    (dict(eps=float("nan")), SHAPE), (dict(eps=float("inf")), SHAPE), (dict(dtype=3), UNSUPPORTED),
    (dict(dtype=-1), UNSUPPORTED), (dict(act=4), UNSUPPORTED), (dict(act=-1), UNSUPPORTED), (dict(xl=2), UNSUPPORTED),
    (dict(yl=-1), UNSUPPORTED),
]


@pytest.mark.parametrize("kw,expect", BAD_NORM, ids=str)
def test_norm_descriptors_are_refused(lib, kw, expect):
    d = norm_desc(**kw)
    out = ctypes.c_size_t(7)
    p = [ctypes.c_void_p(0x100000 * (i + 1)) for i in range(10)]
    for op in (0, 3):
        assert lib.wtconv_group_norm_workspace_size(ctypes.byref(d), op, ctypes.byref(out)) == expect
    assert out.value == 7
    assert lib.wtconv_group_norm_forward(ctypes.byref(d), *p[:6], p[6], 1 << 40, None) == expect
    assert lib.wtconv_group_norm_backward(ctypes.byref(d), *p[:9], p[9], 1 << 40, None) == expect


def test_norm_arguments_are_refused(lib):
    d = norm_desc()
    n = 2 * 8 * 16 * 4  # bytes of an activation
    x, y, dy, st, ws = 0x100000, 0x200000, 0x300000, 0x400000, 0x500000
    out = ctypes.c_size_t(0)
    for op in (1, 2, 4):
        assert lib.wtconv_group_norm_workspace_size(ctypes.byref(d), op, ctypes.byref(out)) == UNSUPPORTED
    assert lib.wtconv_group_norm_workspace_size(ctypes.byref(d), 0, None) == NULL
    assert lib.wtconv_group_norm_workspace_size(None, 0, ctypes.byref(out)) == NULL
    assert lib.wtconv_group_norm_workspace_size(ctypes.byref(d), 3, ctypes.byref(out)) == OK
    need = out.value

    def fwd(x=x, gamma=None, beta=None, y=y, mean=st, rstd=st + 256, ws=ws, nbytes=1 << 30):
        return lib.wtconv_group_norm_forward(ctypes.byref(d), x, gamma, beta, y, mean, rstd, ws, nbytes, None)

    def bwd(x=x, dy=dy, gamma=None, beta=None, mean=st, rstd=st + 256, dx=y, dgamma=st + 512, dbeta=st + 768, ws=ws,
            nbytes=1 << 30):
        return lib.wtconv_group_norm_backward(ctypes.byref(d), x, dy, gamma, beta, mean, rstd, dx, dgamma, dbeta, ws,
                                              nbytes, None)

    for k in ("x", "y", "mean", "rstd"):
        assert fwd(**{k: None}) == NULL
    for k in ("x", "dy", "mean", "rstd", "dx"):
        assert bwd(**{k: None}) == NULL
    for k in ("x", "y", "gamma", "beta", "mean", "rstd"):
        assert fwd(**{k: 0x900002}) == UNSUPPORTED
    for k in ("x", "dy", "dx", "gamma", "beta", "mean", "rstd", "dgamma", "dbeta"):
        assert bwd(**{k: 0x900002}) == UNSUPPORTED
    assert fwd(y=x) == ALIAS and fwd(y=x + n - 4) == ALIAS and fwd(mean=y) == ALIAS and fwd(rstd=st) == ALIAS
    assert fwd(gamma=y + 8) == ALIAS
    assert bwd(dx=x) == ALIAS and bwd(dx=dy + 16) == ALIAS and bwd(dgamma=st) == ALIAS and bwd(dbeta=st + 512) == ALIAS
    assert bwd(ws=dy) == ALIAS
    assert bwd(nbytes=need - 1) == WORKSPACE and bwd(ws=None) == WORKSPACE
    assert bwd(ws=ws + 16) == UNSUPPORTED


BAD_ORTHO = [
    (dict(batch=0), SHAPE), (dict(batch=65536), SHAPE), (dict(rows=0), SHAPE), (dict(cols=-3), SHAPE),
    (dict(rows=1 << 16, cols=1 << 16), SHAPE), (dict(rows=16385, cols=16385), SHAPE), (dict(cols=1 << 62), SHAPE),
    (dict(rows=1, cols=(1 << 22) + 1), SHAPE), (dict(steps=0), SHAPE), (dict(steps=17), SHAPE),
    (dict(batch=65535, rows=1025, cols=1025), SHAPE), (dict(batch=65535, rows=1, cols=1 << 15), SHAPE),
    (dict(eps=-1e-9), SHAPE), (dict(eps=float("nan")), SHAPE), (dict(eps=float("inf")), SHAPE),
    (dict(dtype=3), UNSUPPORTED), (dict(dtype=-1), UNSUPPORTED),
]


@pytest.mark.parametrize("kw,expect", BAD_ORTHO, ids=str)
def test_ortho_descriptors_are_refused(lib, kw, expect):
    d = ortho_desc(**kw)
    h = _native.MuonHyper(0.1, 0.9, 0.0, 1.0, 1)
    out = ctypes.c_size_t(7)
    assert lib.wtconv_orthogonalize_workspace_size(ctypes.byref(d), ctypes.byref(out)) == expect and out.value == 7
    p = [0x10000000 * (i + 1) for i in range(6)]
    assert lib.wtconv_orthogonalize(ctypes.byref(d), p[0], p[1], p[2], 1 << 40, None) == expect
    assert lib.wtconv_muon_step(ctypes.byref(d), ctypes.byref(h), *p, 1 << 40, None) == expect


def test_ortho_arguments_are_refused(lib):
    d = ortho_desc()
    n = 80 * 120 * 4
    need = ctypes.c_size_t(0)
    assert lib.wtconv_orthogonalize_workspace_size(None, ctypes.byref(need)) == NULL
    assert lib.wtconv_orthogonalize_workspace_size(ctypes.byref(d), None) == NULL
    assert lib.wtconv_orthogonalize_workspace_size(ctypes.byref(d), ctypes.byref(need)) == OK
    need = need.value
    big = 1 << 30

    # matrices that one workgroup holds need none
    small = ortho_desc(rows=25, cols=384)
    size = ctypes.c_size_t(7)
    assert lib.wtconv_orthogonalize_workspace_size(ctypes.byref(small), ctypes.byref(size)) == OK and size.value == 0

    def ortho(g=0x100000, out=0x200000, ws=0x1000000, nbytes=big):
        return lib.wtconv_orthogonalize(ctypes.byref(d), g, out, ws, nbytes, None)

    def muon(w=0x100000, g=0x200000, m=0x300000, wo=0x400000, mo=0x500000, ws=0x1000000, nbytes=big, nest=1, h=True):
        hyper = _native.MuonHyper(0.1, 0.9, 0.0, 1.0, nest)
        return lib.wtconv_muon_step(ctypes.byref(d), ctypes.byref(hyper) if h else None, w, g, m, wo, mo, ws, nbytes,
                                    None)

    assert ortho(g=None) == NULL and ortho(out=None) == NULL and ortho(ws=None) == WORKSPACE
    assert ortho(nbytes=need - 1) == WORKSPACE and ortho(ws=0x1000010) == UNSUPPORTED
    assert ortho(g=0x100002) == UNSUPPORTED and ortho(out=0x200001) == UNSUPPORTED
    assert ortho(out=0x100000) == ALIAS and ortho(out=0x100000 + n - 4) == ALIAS
    assert ortho(ws=0x100000) == ALIAS and ortho(ws=0x200000 - 256) == ALIAS
    for k in ("w", "g", "m", "wo", "mo"):
        assert muon(**{k: None}) == NULL and muon(**{k: 0x600002}) == UNSUPPORTED
    assert muon(h=False) == NULL and muon(nest=2) == UNSUPPORTED
    assert muon(ws=None) == WORKSPACE and muon(nbytes=need - 1) == WORKSPACE
    assert muon(wo=0x100000 + 16) == ALIAS and muon(mo=0x300000 - 16) == ALIAS  # neither in place nor apart
    assert muon(wo=0x300000) == ALIAS and muon(mo=0x100000) == ALIAS and muon(wo=0x200000) == ALIAS
    assert muon(mo=0x400000 + 64) == ALIAS and muon(ws=0x500000) == ALIAS and muon(ws=0x200000) == ALIAS


PLAN_SWEEP = """
import ctypes
from level_haar_wavelet_amd import _native
lib = _native.load()
out = ctypes.c_size_t(0)
calls = 0
for c in list(range(1, 18)) + [24, 33, 100, 1030]:
    for h, w in ((1, 1), (1, 7), (2, 2), (3, 5), (4, 6), (8, 8), (16, 16), (17, 16), (37, 23), (64, 64), (256, 128)):
        for groups in {1, c, c // 2 if c % 2 == 0 else 1}:
            for n in (1, 5, 300):
                for dtype in range(3):
                    for xl, yl in ((0, 0), (0, 1), (1, 0), (1, 1)):
                        for op in (_native.OP_FWD, _native.OP_BWD):
                            d = _native.NormDesc(n, c, h, w, groups, dtype, 0, xl, yl, 1e-5)
                            case = (c, h, w, groups, n, dtype, xl, yl, op)
                            out.value = 1 << 62
                            st = lib.wtconv_group_norm_workspace_size(ctypes.byref(d), op, ctypes.byref(out))
                            assert st == 0, case
                            # partial sums of at most the tensor's own size and the last ranges', and means
                            assert out.value <= 8 * n * c * h * w + 8 * n * groups + 1024, (case, out.value)
                            calls += 1
print(calls)
"""


def test_every_small_norm_has_a_plan():
    """Channels fewer than an access has elements, planes it does and does not
    divide, all layouts: in a process of its own, which a fault of the host's
    arithmetic would end."""
    r = subprocess.run([sys.executable, "-c", PLAN_SWEEP], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, (r.returncode, r.stderr[-2000:])
    assert int(r.stdout) > 40000


def test_the_layer_refuses_bf16(lib):
    d = _native.desc(2, 8, 16, 16, 5, 2, _native.BF16)
    out = ctypes.c_size_t(0)
    assert lib.wtconv_workspace_size(ctypes.byref(d), 0, ctypes.byref(out)) == UNSUPPORTED


def test_binding_refuses_cpu_tensors_and_wrong_names():
    x = torch.zeros(2, 8, 4, 4)
    with pytest.raises(TypeError, match="GPU tensor"):
        wt.wtconv_group_norm_forward(x, 2)
    with pytest.raises(TypeError, match="GPU tensor"):
        wt.wtconv_orthogonalize(torch.zeros(4, 4))
    with pytest.raises(TypeError, match="GPU tensor"):
        wt.wtconv_muon_step(torch.zeros(4, 4), torch.zeros(4, 4), torch.zeros(4, 4), lr=0.1)


def test_optimizer_takes_matrices_only():
    from level_haar_wavelet_amd.optim import Muon, _matrices

    assert _matrices((96, 5, 5), None) == (1, 96, 25)
    assert _matrices((3, 384, 5, 5), None) == (3, 384, 25)
    assert _matrices((3, 384, 5, 5), 0) == (1, 3, 384 * 25)
    assert _matrices((8, 12), None) == (1, 8, 12)
    with pytest.raises(ValueError):
        Muon([torch.nn.Parameter(torch.zeros(8))])
    with pytest.raises(TypeError):
        Muon([torch.nn.Parameter(torch.zeros(8, 8, dtype=torch.float16))])
    with pytest.raises(ValueError):
        Muon([torch.nn.Parameter(torch.zeros(8, 8))], lr=-1)


def test_norm_module_checks_its_groups():
    from level_haar_wavelet_amd.module import GroupNormAct2d

    with pytest.raises(ValueError):
        GroupNormAct2d(3, 8)
    m = GroupNormAct2d(4, 8, act="gelu", channels_last=True)
    assert "gelu" in repr(m) and m.gamma.shape == (8,)
    assert GroupNormAct2d(4, 8, affine=False).gamma is None


def test_optimizer_asks_how_an_ordinary_4d_weight_is_meant():
    """(out, in, k, k) of a convolution and (L, 4C, k, k) of the layer look alike:
    only the layer's own parameter, which says so, is a stack by itself."""
    import copy
    import io

    from level_haar_wavelet_amd.module import WTConv2d
    from level_haar_wavelet_amd.optim import Muon

    for k in (1, 3):
        conv = torch.nn.Conv2d(16, 64, k)
        with pytest.raises(ValueError, match="batch_dims"):
            Muon([conv.weight])
        opt = Muon([torch.nn.Parameter(torch.zeros(4, 4))])
        with pytest.raises(ValueError, match="batch_dims"):
            opt.add_param_group({"params": [conv.weight]})
        assert len(opt.param_groups) == 1
        Muon([conv.weight], batch_dims=0)
        Muon([{"params": [conv.weight], "batch_dims": 1}])
        # options of another optimiser's state do not bring the guess back
        opt = Muon([conv.weight], batch_dims=0)
        state = opt.state_dict()
        state["param_groups"][0]["batch_dims"] = None
        opt.load_state_dict(state)
        conv.weight.grad = torch.zeros_like(conv.weight)
        with pytest.raises(ValueError, match="batch_dims"):
            opt.step()
    layer = WTConv2d(4, 3, 2)
    buf = io.BytesIO()
    torch.save(layer, buf)
    buf.seek(0)
    for m in (layer, copy.deepcopy(layer), torch.load(buf, weights_only=False), layer.double().float()):
        Muon([m.w_base, m.w_lvl])
    Muon([WTConv2d(4, 3, 0).w_base])


@pytest.mark.parametrize("kw", [dict(lr=-0.1), dict(lr=float("nan")), dict(momentum=1.0), dict(momentum=-0.1),
                                dict(weight_decay=-1.0), dict(steps=0), dict(steps=17), dict(eps=-1.0),
                                dict(eps=float("inf"))], ids=str)
def test_optimizer_checks_the_options_of_every_group(kw):
    from level_haar_wavelet_amd.optim import Muon

    p = [torch.nn.Parameter(torch.zeros(4, 4)) for _ in range(2)]
    with pytest.raises(ValueError):
        Muon(p, **kw)
    with pytest.raises(ValueError):
        Muon([dict(params=p, **kw)])
    opt = Muon(p[:1])
    with pytest.raises(ValueError):
        opt.add_param_group(dict(params=p[1:], **kw))
    assert len(opt.param_groups) == 1


def test_optimizer_refuses_empty_matrices():
    from level_haar_wavelet_amd.optim import Muon

    for shape in ((0, 4), (4, 0), (2, 0, 3)):
        with pytest.raises(ValueError):
            Muon([torch.nn.Parameter(torch.zeros(shape))])


def test_norm_module_checks_its_options_and_its_input():
    from level_haar_wavelet_amd.module import GroupNormAct2d

    with pytest.raises(ValueError):
        GroupNormAct2d(4, 8, act="tanh")
    for eps in (0.0, -1.0, float("nan"), float("inf")):
        with pytest.raises(ValueError):
            GroupNormAct2d(4, 8, eps=eps)
    for affine in (True, False):  # 16 channels fall into 4 groups too, but are not the module's
        m = GroupNormAct2d(4, 8, affine=affine)
        for shape in ((1, 16, 2, 2), (8, 2, 2), (1, 8, 4)):
            with pytest.raises(ValueError, match="channels"):
                m(torch.zeros(shape))
