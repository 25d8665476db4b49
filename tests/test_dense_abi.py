"""Refusals of the dense operators, in the C ABI and in the binding. Every
call here returns before a kernel is launched, so no GPU is needed: addresses
are only looked at for presence and alignment."""
import pytest
import torch

import mxfp4_routed_expert_sigmoid_amd as k3

A = 0x10000000
OK, INVALID, SHAPE, ALIGN = 0, 1, 3, 4


def _norm(**kw):
    a = dict(h=A, hs=64, d=A + 0x1000, dk=k3.ADD_BF16, ds=64, T=2, H=64, gamma=A + 0x2000, eps=1e-5, x=A + 0x3000,
             xs=64, q=None, qs_=0, s=None, ss=0)
    a.update(kw)
    return k3.lib().k3moe_add_norm(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), INVALID), (dict(H=0), INVALID), (dict(eps=0.0), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(eps=float("inf")), INVALID), (dict(h=None), INVALID), (dict(gamma=None), INVALID),
    (dict(x=None), INVALID), (dict(q=A), INVALID), (dict(s=A), INVALID), (dict(dk=k3.ADD_NONE), INVALID),
    (dict(dk=3), INVALID), (dict(d=None), INVALID), (dict(hs=63), INVALID), (dict(ds=63), INVALID),
    (dict(xs=63), INVALID), (dict(q=A, qs_=64, s=A, ss=1), INVALID), (dict(q=A, qs_=63, s=A, ss=2), INVALID),
    (dict(h=A + 2), ALIGN), (dict(gamma=A + 2), ALIGN), (dict(d=A + 1), ALIGN),
    (dict(d=A + 2, dk=k3.ADD_F32), ALIGN), (dict(x=A + 1), ALIGN), (dict(T=0, h=None), OK),
])
def test_add_norm_refusals(kw, status):
    assert _norm(**kw) == status


def test_add_norm_refuses_rows_that_32_bits_do_not_count():
    """Columns are counted in 32 bits, a block's steps behind the last one included."""
    big = 2 ** 31 - 1
    assert _norm(H=2 ** 30 + 1, hs=big, ds=big, xs=big) == SHAPE
    assert _norm(H=big, hs=big, ds=big, xs=big) == SHAPE


def _linear(**kw):
    a = dict(p=A, s=A + 0x1000, N=32, K=64, x=A + 0x2000, xst=64, xs=None, xsst=0, T=2, out=A + 0x3000, ost=32,
             outs=None, osst=0, kind=k3.OUT_BF16)
    a.update(kw)
    return k3.lib().k3moe_linear(*a.values(), None)


def _glu(act=k3.ACT_SITU, b1=4.0, b2=25.0, up=A + 0x4000, us=A + 0x5000, **kw):
    a = dict(p=A, s=A + 0x1000, up=up, us=us, N=32, K=64, x=A + 0x2000, xst=64, xs=None, xsst=0, T=2, act=act,
             b1=b1, b2=b2, out=A + 0x3000, ost=32, outs=None, osst=0, kind=k3.OUT_BF16)
    a.update(kw)
    return k3.lib().k3moe_glu(*a.values(), None)


DENSE = [
    (dict(T=-1), INVALID), (dict(N=0), INVALID), (dict(K=0), INVALID), (dict(K=48), SHAPE), (dict(K=16), SHAPE),
    (dict(kind=0), INVALID), (dict(kind=5), INVALID), (dict(p=None), INVALID), (dict(s=None), INVALID),
    (dict(x=None), INVALID), (dict(out=None), INVALID), (dict(outs=A), INVALID),
    (dict(kind=k3.OUT_MXFP8), INVALID), (dict(xst=56), INVALID), (dict(ost=31), INVALID),
    (dict(xs=A, xsst=1), INVALID), (dict(kind=k3.OUT_MXFP8, outs=A, osst=0), INVALID),
    (dict(p=A + 8), ALIGN), (dict(s=A + 4), ALIGN), (dict(x=A + 8), ALIGN), (dict(xst=68), ALIGN),
    (dict(xs=A, xsst=2, xst=72), ALIGN), (dict(out=A + 1), ALIGN), (dict(out=A + 2, kind=k3.OUT_F32), ALIGN),
    (dict(xst=2 ** 24 + 16), SHAPE), (dict(xs=A, xsst=2, xst=2 ** 24 + 16), SHAPE),
    (dict(T=0, x=None, out=None), OK),
]


@pytest.mark.parametrize("kw,status", DENSE)
def test_linear_refusals(kw, status):
    assert _linear(**kw) == status


@pytest.mark.parametrize("kw,status", DENSE + [
    (dict(act=0), INVALID), (dict(act=3), INVALID), (dict(b1=0.0), INVALID), (dict(b2=float("inf")), INVALID),
    (dict(b2=float("nan")), INVALID), (dict(up=None), INVALID), (dict(us=None), INVALID), (dict(up=A + 8), ALIGN),
    (dict(kind=k3.OUT_F32_ADD), INVALID), (dict(act=k3.ACT_SWIGLU, b1=0.0, T=0), OK),
])
def test_glu_refusals(kw, status):
    assert _glu(**kw) == status


def test_grids_beyond_32_bits_are_refused():
    big = dict(T=2 ** 31 - 1, N=2 ** 31 - 1, ost=2 ** 31 - 1)
    assert _linear(**big) == SHAPE and _glu(**big) == SHAPE


class _Dev:
    """Stands in for a device tensor where only shape, type and strides are looked at."""

    def __init__(self, t, device="cuda:0"):
        self.t, self.is_cuda, self.device = t, True, torch.device(device)

    def __getattr__(self, n):
        return getattr(self.t, n)

    def get_device(self):
        return self.device.index


def _z(*shape, dtype=torch.float32):
    return _Dev(torch.zeros(shape, dtype=dtype))


def test_binding_refuses_wrong_tensors_of_add_norm(monkeypatch):
    monkeypatch.setattr(k3, "lib", lambda: pytest.fail("the library was reached"))
    bf, u8 = torch.bfloat16, torch.uint8
    good = dict(h=_z(3, 70), gamma=_z(70), eps=1e-5, d=_z(3, 70, dtype=bf), x=_z(3, 70, dtype=bf),
                q=_z(3, 70, dtype=u8), qs=_z(3, 3, dtype=u8))
    wide = _Dev(torch.zeros(70, 3).t())                        # rows are not contiguous
    over = _Dev(torch.zeros(400).as_strided((3, 70), (35, 1)))  # rows overlap
    for bad in (dict(h=_z(70)), dict(h=_z(3, 70, dtype=bf)), dict(h=wide), dict(h=over), dict(gamma=_z(71)),
                dict(gamma=_z(70, dtype=bf)), dict(d=_z(2, 70)), dict(d=_z(3, 70, dtype=torch.float16)),
                dict(x=_z(3, 70)), dict(q=_z(3, 70, dtype=torch.float8_e5m2)), dict(qs=_z(3, 2, dtype=u8)),
                dict(q=None), dict(qs=None), dict(x=torch.zeros(3, 70, dtype=bf)),
                dict(d=_Dev(torch.zeros(3, 70), "cuda:1"))):
        with pytest.raises(ValueError):
            k3.add_norm(**{**good, **bad})


def test_binding_refuses_wrong_tensors_of_the_products(monkeypatch):
    monkeypatch.setattr(k3, "lib", lambda: pytest.fail("the library was reached"))
    bf, u8 = torch.bfloat16, torch.uint8
    good = dict(packed=_z(40, 32, dtype=u8), scales=_z(40, 2, dtype=u8), x=_z(3, 64, dtype=bf),
                out=_z(3, 40, dtype=bf))
    bads = [dict(packed=_z(40, 24, dtype=u8)), dict(packed=_z(40, 32)), dict(scales=_z(40, 3, dtype=u8)),
            dict(x=_z(3, 96, dtype=bf)), dict(x=_z(3, 64)), dict(x=_z(3, 64, dtype=u8)),
            dict(xs=_z(3, 2, dtype=u8)), dict(out=_z(2, 40, dtype=bf)), dict(out=_z(3, 40, dtype=torch.float64)),
            dict(outs=_z(3, 2, dtype=u8)), dict(out=_z(3, 40, dtype=u8), outs=_z(3, 1, dtype=u8)),
            dict(x=torch.zeros(3, 64, dtype=bf)), dict(scales=_Dev(torch.zeros(40, 2, dtype=u8), "cuda:1"))]
    for bad in bads + [dict(accumulate=True), dict(out=_z(3, 40, dtype=u8), outs=_z(3, 2, dtype=u8), accumulate=True)]:
        with pytest.raises(ValueError):
            k3.linear(**{**good, **bad})
    for bad in bads + [dict(up_packed=_z(39, 32, dtype=u8))]:
        v = {**good, **bad}
        with pytest.raises(ValueError):
            k3.glu(v["packed"], v["scales"], v.get("up_packed", good["packed"]), good["scales"], v["x"], v["out"],
                   xs=v.get("xs"), outs=v.get("outs"))


def test_binding_refuses_sizes_past_32_bits(monkeypatch):
    """A row count would be cut to its low 32 bits on its way into the library."""
    monkeypatch.setattr(k3, "lib", lambda: pytest.fail("the call was made"))
    wide = torch.empty(1, 32).expand(2 ** 32 + 2, 32)
    with pytest.raises(ValueError, match="counted in 32 bits"):
        k3.add_norm(wide, _z(32), 1e-5, x=wide)
    x = torch.empty(1, 32, dtype=torch.bfloat16).expand(2 ** 32 + 2, 32)
    w, s = _z(32, 16, dtype=torch.uint8), _z(32, 1, dtype=torch.uint8)
    with pytest.raises(ValueError):
        k3.linear(w, s, x, x)


def test_numbers_agree_with_the_header():
    import os
    import re
    from conftest import ROOT
    src = open(os.path.join(ROOT, "include", "k3moe.h")).read()
    for name in ("ADD_NONE", "ADD_BF16", "ADD_F32", "OUT_BF16", "OUT_F32", "OUT_F32_ADD", "OUT_MXFP8"):
        assert int(re.search(rf"K3MOE_{name} = (\d)", src).group(1)) == getattr(k3, name)
