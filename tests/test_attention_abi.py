"""Refusals of the attention operators and of those around them, in the C ABI
and in the binding. Every call here returns before a kernel is launched, so no
GPU is needed: addresses are only looked at for presence and alignment."""
import ctypes
import os
import re

import pytest
import torch

import mxfp4_routed_expert_sigmoid_amd as k3
from test_dense_abi import _Dev, _z

A = 0x10000000
OK, INVALID, SHAPE, ALIGN, WORKSPACE = 0, 1, 3, 4, 5
BIG = 2 ** 31 - 1


def _pages(k=A, v=A, ks=None, vs=None, pages=4, page=16):
    return k3._PAGES(k or 0, v or 0, ks or 0, vs or 0, pages, page)


def _heads(**kw):
    a = dict(q=A, qst=512, k=A, kst=128, v=A, vst=128, T=2, Hq=8, Hkv=2, D=64, Dv=64, gq=A, gk=A, eps=1e-5, pos=A, freq=A,
             R=64, rot=1, qo=A, qost=512, ko=A, kost=128, cache=_pages(), slots=A)
    a.update(kw)
    return k3.lib().k3moe_qk_norm_rope(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), INVALID), (dict(Hq=0), INVALID), (dict(Hkv=0), INVALID), (dict(D=0), INVALID), (dict(R=-2), INVALID),
    (dict(R=128), INVALID), (dict(eps=0.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID),
    (dict(rot=0), INVALID), (dict(rot=3), INVALID), (dict(freq=None), INVALID), (dict(R=0), INVALID),
    (dict(slots=None), INVALID), (dict(v=None), INVALID), (dict(cache=None), INVALID), (dict(Dv=0), INVALID),
    (dict(pos=None), INVALID), (dict(q=None), INVALID), (dict(k=None), INVALID),
    (dict(qo=None, ko=None, cache=None, v=None, slots=None), INVALID), (dict(qst=511), INVALID), (dict(kst=120), INVALID),
    (dict(vst=120), INVALID), (dict(qost=504), INVALID), (dict(kost=120), INVALID), (dict(cache=_pages(k=None)), INVALID),
    (dict(cache=_pages(ks=A)), INVALID), (dict(cache=_pages(vs=A)), INVALID), (dict(cache=_pages(pages=-1)), INVALID),
    (dict(cache=_pages(page=0)), INVALID),
    (dict(cache=_pages(page=8)), SHAPE), (dict(cache=_pages(page=48)), SHAPE), (dict(cache=_pages(page=2 ** 21)), SHAPE),
    (dict(D=60, R=0, freq=None), SHAPE), (dict(D=264, R=0, freq=None), SHAPE), (dict(R=24), SHAPE), (dict(Dv=60), SHAPE),
    (dict(Dv=264), SHAPE), (dict(Hq=4097), SHAPE), (dict(Hkv=4097), SHAPE), (dict(T=2 ** 25 + 1), SHAPE),
    (dict(cache=_pages(ks=A, vs=A), Dv=40), SHAPE), (dict(cache=_pages(ks=A, vs=A), D=40, R=16), SHAPE),
    (dict(q=A + 8), ALIGN), (dict(k=A + 8), ALIGN), (dict(v=A + 8), ALIGN), (dict(qo=A + 8), ALIGN), (dict(ko=A + 8), ALIGN),
    (dict(qst=516), ALIGN), (dict(kst=132), ALIGN), (dict(vst=132), ALIGN), (dict(qost=516), ALIGN), (dict(kost=132), ALIGN),
    (dict(gq=A + 2), ALIGN), (dict(gk=A + 2), ALIGN), (dict(pos=A + 2), ALIGN), (dict(freq=A + 2), ALIGN),
    (dict(slots=A + 4), ALIGN), (dict(cache=_pages(k=A + 8)), ALIGN), (dict(cache=_pages(v=A + 8)), ALIGN),
    (dict(T=0, q=None, k=None, v=None, slots=None), OK),
    (dict(qo=None, ko=None, cache=_pages(pages=0, k=None, v=None)), OK),
])
def test_qk_norm_rope_refusals(kw, status):
    assert _heads(**kw) == status


def _att(**kw):
    a = dict(q=A, qst=512, k=A, kst=128, v=A, vst=128, cq=A, ck=A, seqs=2, Tq=9, Tk=9, Hq=8, Hkv=2, D=64, Dv=64, scale=0.125,
             causal=1, out=A, ost=512, lse=A, ws=None, n=0)
    a.update(kw)
    return k3.lib().k3moe_attention(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(seqs=-1), INVALID), (dict(Tq=-1), INVALID), (dict(Tk=-1), INVALID), (dict(Hq=0), INVALID), (dict(Hkv=0), INVALID),
    (dict(Hq=7), INVALID), (dict(causal=2), INVALID), (dict(causal=-1), INVALID), (dict(scale=0.0), INVALID),
    (dict(scale=-1.0), INVALID), (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(cq=None), INVALID),
    (dict(out=None), INVALID), (dict(qst=504), INVALID), (dict(kst=120), INVALID), (dict(vst=120), INVALID),
    (dict(ost=504), INVALID), (dict(D=96, Dv=96), SHAPE), (dict(D=128), SHAPE), (dict(D=192), SHAPE), (dict(Dv=128), SHAPE),
    (dict(qst=2 ** 24 + 8), SHAPE), (dict(kst=2 ** 24 + 8), SHAPE), (dict(vst=2 ** 24 + 8), SHAPE),
    (dict(ost=2 ** 24 + 8), SHAPE), (dict(Tq=BIG, seqs=BIG), SHAPE), (dict(Tq=BIG, seqs=1), SHAPE),
    (dict(q=A + 8), ALIGN), (dict(k=A + 2), ALIGN), (dict(v=A + 8), ALIGN), (dict(out=A + 8), ALIGN), (dict(qst=516), ALIGN),
    (dict(kst=132), ALIGN), (dict(vst=132), ALIGN), (dict(ost=516), ALIGN), (dict(cq=A + 2), ALIGN), (dict(ck=A + 2), ALIGN),
    (dict(scale=3e19), INVALID), (dict(seqs=2 ** 30 + 1), SHAPE),
    (dict(lse=A + 2), ALIGN), (dict(ws=A + 128, n=1 << 30), WORKSPACE), (dict(ws=A, Tk=9000, n=100), WORKSPACE),
    (dict(ws=A, Tk=9000, n="short"), WORKSPACE), (dict(seqs=0), OK), (dict(Tq=0, q=None, out=None, cq=None), OK),
])
def test_attention_refusals(kw, status):
    if kw.get("n") == "short":
        kw = dict(kw, n=k3._attention_bytes(2, 9, 9000, 8, 64) - 1)
    assert _att(**kw) == status


def test_attention_workspace_refusals():
    n, m = ctypes.c_size_t(), ctypes.c_size_t()
    f = k3.lib().k3moe_attention_workspace_size
    assert f(1, 100, 9000, 8, 128, ctypes.byref(n)) == OK and n.value > 0
    assert f(2, 9, 800, 64, 128, ctypes.byref(m)) == OK and m.value in (0, n.value)   # one size serves every call
    assert f(1, 1, 40000, 1, 128, ctypes.byref(m)) == OK and m.value == n.value
    assert f(1, 100, 100, 8, 128, ctypes.byref(n)) == OK and n.value == 0        # nothing to split
    assert f(BIG, BIG, BIG, BIG, 128, ctypes.byref(n)) == OK and n.value == 0
    assert f(0, 0, 0, 1, 64, ctypes.byref(n)) == OK and n.value == 0
    for a, want in (((-1, 1, 1, 1, 64), INVALID), ((1, -1, 1, 1, 64), INVALID), ((1, 1, -1, 1, 64), INVALID),
                    ((1, 1, 1, 0, 64), INVALID), ((1, 1, 1, 1, 96), SHAPE)):
        assert f(*a, ctypes.byref(n)) == want
    assert f(1, 1, 1, 1, 64, None) == INVALID


def _tree(**kw):
    a = dict(q=A, qst=512, cache=_pages(), pages=A, width=4, lens=A, cq=A, tree=A, seqs=2, Tq=4, maxq=2, Hq=8, Hkv=2, D=64,
             Dv=64, scale=0.125, out=A, ost=512, lse=A, ws=A, n=1 << 30)
    a.update(kw)
    return k3.lib().k3moe_tree_attention(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(cache=None), INVALID), (dict(seqs=-1), INVALID), (dict(Tq=-1), INVALID), (dict(maxq=0), INVALID),
    (dict(Hq=0), INVALID), (dict(Hkv=0), INVALID), (dict(Hq=7), INVALID), (dict(width=-1), INVALID),
    (dict(cache=_pages(pages=-1)), INVALID), (dict(cache=_pages(page=0)), INVALID), (dict(scale=0.0), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID), (dict(cq=None, Tq=5), INVALID),
    (dict(scale=3e19), INVALID),
    (dict(cq=None, maxq=1), INVALID), (dict(q=None), INVALID), (dict(lens=None), INVALID), (dict(out=None), INVALID),
    (dict(pages=None), INVALID), (dict(cache=_pages(ks=A)), INVALID), (dict(cache=_pages(vs=A)), INVALID),
    (dict(cache=_pages(k=None)), INVALID), (dict(cache=_pages(v=None)), INVALID), (dict(qst=504), INVALID),
    (dict(ost=504), INVALID), (dict(D=96, Dv=96), SHAPE), (dict(D=128), SHAPE), (dict(maxq=65), SHAPE),
    (dict(cache=_pages(page=8)), SHAPE), (dict(cache=_pages(page=40)), SHAPE), (dict(cache=_pages(page=2 ** 21)), SHAPE),
    (dict(width=2 ** 26 + 1), SHAPE), (dict(seqs=2 ** 30, Tq=2 ** 30), SHAPE), (dict(seqs=2 ** 20, Tq=2 ** 20, width=2 ** 20), SHAPE),
    (dict(q=A + 8), ALIGN), (dict(out=A + 8), ALIGN), (dict(qst=516), ALIGN), (dict(ost=516), ALIGN), (dict(pages=A + 2), ALIGN), (dict(lens=A + 2), ALIGN),
    (dict(cq=A + 2), ALIGN), (dict(tree=A + 4), ALIGN), (dict(lse=A + 2), ALIGN), (dict(cache=_pages(k=A + 8)), ALIGN),
    (dict(cache=_pages(v=A + 8)), ALIGN), (dict(ws=None), WORKSPACE), (dict(ws=A + 128), WORKSPACE), (dict(n=0), WORKSPACE),
    (dict(n="short"), WORKSPACE), (dict(seqs=0), OK), (dict(Tq=0, q=None, out=None), OK),
])
def test_tree_attention_refusals(kw, status):
    if kw.get("n") == "short":
        kw = dict(n=k3._tree_bytes(8, 2, 64, 2) - 1)
    assert _tree(**kw) == status


def test_tree_attention_workspace_refusals():
    n = ctypes.c_size_t()
    f = k3.lib().k3moe_tree_attention_workspace_size
    assert f(8, 2, 128, 1, ctypes.byref(n)) == OK and n.value > 0
    for a, want in (((0, 2, 128, 1), INVALID), ((8, 3, 128, 1), INVALID), ((8, 0, 128, 1), INVALID), ((8, 2, 128, 0), INVALID),
                    ((8, 2, 96, 1), SHAPE), ((8, 2, 128, 65), SHAPE), ((8192, 2, 128, 1), SHAPE)):
        assert f(*a, ctypes.byref(n)) == want
    assert f(8, 2, 128, 1, None) == INVALID


def _lp(**kw):
    a = dict(x=A, f32=1, st=100, T=2, V=100, ids=A, M=1, lp=A, ent=A, ti=A, tl=A, k=3, ws=A, n=1 << 30)
    a.update(kw)
    return k3.lib().k3moe_logprobs(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(f32=2), INVALID), (dict(f32=-1), INVALID), (dict(M=-1), INVALID), (dict(T=-1), INVALID), (dict(V=0), INVALID),
    (dict(k=-1), INVALID), (dict(k=101), INVALID), (dict(x=None), INVALID), (dict(ids=None), INVALID), (dict(lp=None), INVALID),
    (dict(M=0), INVALID), (dict(ti=None), INVALID), (dict(tl=None), INVALID), (dict(k=0), INVALID), (dict(st=99), INVALID),
    (dict(ids=None, M=0, lp=None, ent=None, ti=None, tl=None, k=0), INVALID), (dict(V=2 ** 24 + 1, st=BIG), SHAPE),
    (dict(k=65), SHAPE), (dict(M=4097), SHAPE), (dict(T=2 ** 24), SHAPE), (dict(x=A + 2), ALIGN), (dict(x=A + 1, f32=0), ALIGN),
    (dict(ids=A + 2), ALIGN), (dict(lp=A + 1), ALIGN), (dict(ent=A + 2), ALIGN), (dict(ti=A + 2), ALIGN),
    (dict(tl=A + 2), ALIGN), (dict(ws=None), WORKSPACE), (dict(ws=A + 16), WORKSPACE), (dict(n=10), WORKSPACE),
    (dict(n="short"), WORKSPACE), (dict(T=0, x=None), OK),
])
def test_logprobs_refusals(kw, status):
    if kw.get("n") == "short":
        kw = dict(n=k3._logprobs_bytes(2, 100, 3) - 1)
    assert _lp(**kw) == status


def test_logprobs_workspace_refusals():
    n = ctypes.c_size_t()
    f = k3.lib().k3moe_logprobs_workspace_size
    assert f(2, 100, 3, ctypes.byref(n)) == OK and n.value > 0
    for a, want in (((-1, 100, 3), INVALID), ((2, 0, 0), INVALID), ((2, 100, 101), INVALID), ((2, 100, 65), SHAPE),
                    ((2, 2 ** 24 + 1, 3), SHAPE), ((BIG, 2 ** 24, 3), SHAPE)):
        assert f(*a, ctypes.byref(n)) == want
    assert f(2, 100, 3, None) == INVALID


BF, U8, I32, I64 = torch.bfloat16, torch.uint8, torch.int32, torch.int64


def _refused(call, good, bads):
    for bad in bads:
        with pytest.raises(ValueError):
            call(**{**good, **bad})
            print("accepted", bad)


def test_binding_refuses_wrong_tensors_of_qk_norm_rope(monkeypatch):
    monkeypatch.setattr(k3, "lib", lambda: pytest.fail("the library was reached"))
    q, k, v = _z(3, 4, 64, dtype=BF), _z(3, 2, 64, dtype=BF), _z(3, 2, 32, dtype=BF)
    good = dict(q=q, k=k, positions=_z(3, dtype=I32), inv_freq=_z(32), gamma_q=_z(64), gamma_k=_z(64), q_out=q, k_out=k, v=v,
                kc=_z(5, 2, 16, 64, dtype=BF), vc=_z(5, 2, 16, 32, dtype=BF), slots=_z(3, dtype=I64))
    heads_apart = _Dev(torch.zeros(3, 4, 80, dtype=BF)[:, :, :64])
    over = _Dev(torch.zeros(900, dtype=BF).as_strided((3, 4, 64), (128, 64, 1)))
    _refused(k3.qk_norm_rope, good, [
        dict(q=_z(3, 256, dtype=BF)), dict(q=_z(3, 4, 64)), dict(q=heads_apart), dict(q=over), dict(k=_z(2, 2, 64, dtype=BF)),
        dict(k=_z(3, 2, 32, dtype=BF)), dict(positions=_z(3, dtype=I64)), dict(positions=_z(4, dtype=I32)),
        dict(inv_freq=_z(32, 1)), dict(inv_freq=_z(32, dtype=BF)), dict(gamma_q=_z(63)), dict(gamma_k=_z(64, dtype=BF)),
        dict(q_out=_z(3, 2, 64, dtype=BF)), dict(k_out=_z(3, 2, 64)), dict(v=None), dict(slots=None), dict(kc=None), dict(vc=None),
        dict(v=_z(3, 1, 32, dtype=BF)), dict(kc=_z(5, 2, 16, 32, dtype=BF)), dict(kc=_z(5, 1, 16, 64, dtype=BF)),
        dict(vc=_z(4, 2, 16, 32, dtype=BF)), dict(vc=_z(5, 2, 16, 64, dtype=BF)), dict(kc=_z(5, 2, 16, 64)),
        dict(ks=_z(5, 2, 16, 2, dtype=U8)), dict(ks=_z(5, 2, 16, 2, dtype=U8), vs=_z(5, 2, 16, 1, dtype=U8)),
        dict(slots=_z(3, dtype=I32)), dict(slots=_z(4, dtype=I64)), dict(q=torch.zeros(3, 4, 64, dtype=BF)),
        dict(k=_Dev(torch.zeros(3, 2, 64, dtype=BF), "cuda:1")),
        dict(kc=_Dev(torch.zeros(5, 2, 16, 128, dtype=BF)[..., :64]))])
    with pytest.raises(ValueError):
        k3.qk_norm_rope(q, k, good["positions"], good["inv_freq"], q_out=q, ks=_z(5, 2, 16, 2, dtype=U8))


def test_binding_refuses_wrong_tensors_of_attention(monkeypatch):
    monkeypatch.setattr(k3, "lib", lambda: pytest.fail("the library was reached"))
    good = dict(q=_z(9, 4, 64, dtype=BF), k=_z(9, 2, 64, dtype=BF), v=_z(9, 2, 64, dtype=BF), cu_q=_z(3, dtype=I32),
                out=_z(9, 4, 64, dtype=BF), cu_k=_z(3, dtype=I32), lse=_z(9, 4))
    _refused(k3.attention, good, [
        dict(q=_z(9, 256, dtype=BF)), dict(q=_z(9, 4, 64)), dict(q=_z(9, 3, 64, dtype=BF)), dict(k=_z(8, 2, 64, dtype=BF)),
        dict(k=_z(9, 2, 32, dtype=BF)), dict(v=_z(9, 1, 64, dtype=BF)), dict(v=_z(9, 2, 64)), dict(cu_q=_z(3, dtype=I64)),
        dict(cu_q=_z(0, dtype=I32)), dict(cu_q=_z(3, 1, dtype=I32)), dict(cu_k=_z(2, dtype=I32)), dict(out=_z(9, 4, 32, dtype=BF)),
        dict(out=_z(9, 4, 64)), dict(lse=_z(9, 2)), dict(lse=_z(9, 4, dtype=BF)), dict(q=torch.zeros(9, 4, 64, dtype=BF)),
        dict(cu_q=_Dev(torch.zeros(3, dtype=I32), "cuda:1"))])


def test_binding_refuses_wrong_tensors_of_tree_attention(monkeypatch):
    monkeypatch.setattr(k3, "lib", lambda: pytest.fail("the library was reached"))
    good = dict(q=_z(4, 4, 64, dtype=BF), kc=_z(5, 2, 16, 64, dtype=BF), vc=_z(5, 2, 16, 64, dtype=BF), pages=_z(2, 3, dtype=I32),
                lens=_z(2, dtype=I32), out=_z(4, 4, 64, dtype=BF), cu_q=_z(3, dtype=I32), max_q=2, tree=_z(4, dtype=I64),
                lse=_z(4, 4), workspace=_z(10, dtype=U8))
    _refused(k3.tree_attention, good, [
        dict(q=_z(4, 256, dtype=BF)), dict(q=_z(4, 4, 64)), dict(q=_z(4, 3, 64, dtype=BF)), dict(kc=_z(5, 2, 16, 32, dtype=BF)),
        dict(vc=_z(5, 1, 16, 64, dtype=BF)), dict(vc=_z(4, 2, 16, 64, dtype=BF)), dict(ks=_z(5, 2, 16, 2, dtype=U8)),
        dict(pages=_z(2, dtype=I32)), dict(pages=_z(2, 3, dtype=I64)), dict(lens=_z(3, dtype=I32)), dict(lens=_z(2, dtype=I64)),
        dict(out=_z(4, 4, 32, dtype=BF)), dict(cu_q=_z(2, dtype=I32)), dict(max_q=None), dict(tree=_z(4, dtype=I32)),
        dict(tree=_z(3, dtype=I64)), dict(lse=_z(4, 2)), dict(workspace=_z(10)), dict(q=torch.zeros(4, 4, 64, dtype=BF)),
        dict(pages=_Dev(torch.zeros(2, 3, dtype=I32), "cuda:1"))])


def test_binding_refuses_wrong_tensors_of_logprobs(monkeypatch):
    monkeypatch.setattr(k3, "lib", lambda: pytest.fail("the library was reached"))
    good = dict(logits=_z(3, 50), ids=_z(3, 2, dtype=I32), lp=_z(3, 2), entropy=_z(3), top_ids=_z(3, 4, dtype=I32),
                top_lp=_z(3, 4), workspace=_z(10, dtype=U8))
    _refused(k3.logprobs, good, [
        dict(logits=_z(50)), dict(logits=_z(3, 50, dtype=torch.float16)), dict(logits=_Dev(torch.zeros(50, 3).t())),
        dict(ids=None), dict(lp=None), dict(top_ids=None), dict(top_lp=None), dict(ids=_z(3, 2, dtype=I64)),
        dict(ids=_z(3, dtype=I32)), dict(lp=_z(3, 1)), dict(entropy=_z(3, 1)), dict(entropy=_z(3, dtype=BF)),
        dict(top_ids=_z(3, 3, dtype=I32)), dict(top_lp=_z(3, 4, dtype=BF)), dict(logits=torch.zeros(3, 50)),
        dict(workspace=_Dev(torch.zeros(10, dtype=U8), "cuda:1"))])


def test_binding_refuses_sizes_past_32_bits(monkeypatch):
    """A size would be cut to its low 32 bits on its way into the library."""
    monkeypatch.setattr(k3, "lib", lambda: pytest.fail("the call was made"))
    wide = _Dev(torch.empty(1, 1, 64, dtype=BF).expand(2 ** 32 + 2, 1, 64))
    with pytest.raises(ValueError, match="counted in 32 bits"):
        k3.qk_norm_rope(wide, wide, None, None, q_out=wide)
    with pytest.raises(ValueError, match="counted in 32 bits"):
        k3.attention(wide, wide, wide, _z(2, dtype=I32), wide)
    pool = _Dev(torch.empty(1, 1, 16, 64, dtype=BF).expand(2 ** 32 + 2, 1, 16, 64))
    with pytest.raises(ValueError, match="counted in 32 bits"):
        k3.tree_attention(_z(2, 1, 64, dtype=BF), pool, pool, _z(2, 1, dtype=I32), _z(2, dtype=I32), _z(2, 1, 64, dtype=BF))
    with pytest.raises(ValueError, match="counted in 32 bits"):
        k3.logprobs(_Dev(torch.empty(1, 8).expand(2 ** 32 + 2, 8)), entropy=_z(3))


def _tracked(*shape, dtype=torch.float32):
    t = _z(*shape, dtype=dtype)
    t.t.requires_grad_()
    return t


@pytest.mark.parametrize("i", range(9))
def test_results_that_require_grad_are_refused(monkeypatch, i):
    monkeypatch.setattr(k3, "lib", lambda: pytest.fail("the call was made"))
    q, kv, cu = _z(4, 4, 64, dtype=BF), _z(4, 2, 64, dtype=BF), _z(3, dtype=I32)
    pool, tq, x = _z(5, 2, 16, 64, dtype=BF), _tracked(4, 4, 64, dtype=BF), _z(4, 50)
    cached = dict(v=kv, kc=pool, vc=pool, slots=_z(4, dtype=I64))
    calls = [
        lambda: k3.qk_norm_rope(q, kv, None, None, q_out=tq),
        lambda: k3.qk_norm_rope(q, kv, None, None, k_out=_tracked(4, 2, 64, dtype=BF)),
        lambda: k3.qk_norm_rope(q, kv, None, None, **{**cached, "vc": _tracked(5, 2, 16, 64, dtype=BF)}),
        lambda: k3.attention(q, kv, kv, cu, tq),
        lambda: k3.attention(q, kv, kv, cu, q, lse=_tracked(4, 4)),
        lambda: k3.tree_attention(q, pool, pool, _z(2, 3, dtype=I32), _z(2, dtype=I32), tq),
        lambda: k3.logprobs(x, entropy=_tracked(4)),
        lambda: k3.logprobs(x, ids=_z(4, 1, dtype=I32), lp=_tracked(4, 1)),
        lambda: k3.logprobs(x, top_ids=_z(4, 1, dtype=I32), top_lp=_tracked(4, 1)),
    ]
    with pytest.raises(ValueError, match="requires grad"):
        calls[i]()


def test_numbers_agree_with_the_header():
    from conftest import ROOT
    src = open(os.path.join(ROOT, "include", "k3moe.h")).read()
    for name in ("ROT_HALVES", "ROT_PAIRS"):
        assert int(re.search(rf"K3MOE_{name} = (\d)", src).group(1)) == getattr(k3, name)


@pytest.mark.parametrize("Tq,Tk,H", [(1, 255, 8), (1, 256, 8), (1, 383, 8), (1, 384, 8), (1, 511, 8), (128, 511, 32), (1, 512, 8),
                                     (64, 4096, 32), (1, 8192, 256), (1, 8192, 257), (129, 4096, 128)])
def test_attention_makes_a_workspace_wherever_one_is_used(monkeypatch, Tq, Tk, H):
    """With none given the binding makes one for every call that the library would split with one."""
    made, real = [], k3.lib()

    class Lib:
        k3moe_attention_workspace_size = real.k3moe_attention_workspace_size

        @staticmethod
        def k3moe_attention(*a):
            made.append(a[-3] is not None)
            return OK

    monkeypatch.setattr(k3, "lib", lambda: Lib)
    monkeypatch.setattr(k3, "_elsewhere", lambda dev: False)
    monkeypatch.setattr(k3, "_changed", lambda t: None)
    monkeypatch.setattr(k3, "_queue", lambda dev, stream: 0)
    monkeypatch.setattr(k3, "_scratch", lambda ws, size, device, stream: (ws, A, size()))
    q, kv = _z(Tq, H, 64, dtype=BF), _z(Tk, 1, 64, dtype=BF)
    k3.attention(q, kv, kv, _z(2, dtype=I32), q, cu_k=_z(2, dtype=I32))
    assert made == [k3._attention_bytes(1, Tq, Tk, H, 64) > 0]
