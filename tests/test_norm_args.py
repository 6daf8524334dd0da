"""Host-only checks of the residual norm's arguments (no GPU, nothing launched)."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def coli():
    from int4_routed_expert_bias_b200 import _build
    _build.build()
    import int4_routed_expert_bias_b200 as m
    return m


# far apart, non-null and aligned: argument checks never read through them
D, R, G, RO, Y, W1, W2 = ((i + 1) << 30 for i in range(7))


def _norm(coli, **over):
    kw = dict(hidden=1024, eps=1e-5, post_w=W1, pre_w=W2, gate=0, gate_sigmoid=0, residual_scale=1.0, block_scale=1.0)
    kw.update(over)
    s = coli._BlockNormStruct()
    for k, v in kw.items():
        setattr(s, k, v)
    return s


def _call(coli, n, d=D, xt=1, r=R, rt=1, g=None, T=4, ro=RO, y=Y):
    return coli.lib().coli_residual_norm(ctypes.byref(n) if n is not None else None, d, xt, r, rt, g, T, ro, y, None)


@pytest.mark.parametrize("over", [
    dict(hidden=0), dict(hidden=16385), dict(eps=-1.0), dict(eps=float("nan")), dict(gate=4), dict(gate=-1),
    dict(gate_sigmoid=2), dict(residual_scale=float("inf")), dict(block_scale=float("nan")), dict(post_w=W1 + 4),
    dict(pre_w=W2 + 8), dict(pre_w=None), dict(gate=1)])
def test_bad_norm_is_refused(coli, over):
    assert _call(coli, _norm(coli, **over)) == 1
    assert coli.last_error()


@pytest.mark.parametrize("over", [
    dict(xt=2), dict(rt=-1), dict(T=-1), dict(T=65537), dict(d=None), dict(r=None), dict(y=None), dict(d=D + 4),
    dict(r=R + 2), dict(ro=RO + 8), dict(y=Y + 1), dict(ro=None, y=None),
    dict(ro=D, rt=0),             # same place, another type
    dict(ro=D + 2048), dict(ro=R - 2048), dict(y=R + 16), dict(y=RO), dict(ro=Y - 16), dict(ro=W1), dict(y=W2)])
def test_bad_call_is_refused(coli, over):
    assert _call(coli, _norm(coli), **over) == 1
    assert coli.last_error()


def test_gate_overlaps(coli):
    assert _call(coli, _norm(coli, gate=2), g=G, y=G) == 1
    assert _call(coli, _norm(coli, gate=1), g=G, ro=G) == 1
    assert _call(coli, _norm(coli, gate=3), g=G + 16, y=G) == 1
    assert _call(coli, _norm(coli, gate=3), g=G + 4) == 1


def test_no_block_needs_no_gate_and_no_norm_of_it(coli):
    assert _call(coli, _norm(coli), d=None) == 1
    assert _call(coli, _norm(coli, post_w=None, gate=2), d=None, g=G) == 1
    assert _call(coli, None) == 1


def test_empty_batch(coli):
    assert _call(coli, _norm(coli), T=0) == 0


def test_empty_tensors(coli):
    """Tensors without elements have no address: no pointer is looked at."""
    import torch
    w = torch.ones(64)
    n = coli.BlockNorm(64, post_w=w, pre_w=w, gate="token")
    e = torch.empty(0, 64)
    assert e.data_ptr() == 0
    coli.residual_norm(n, e, e.clone(), e.clone(), e.clone(), gate=torch.empty(0), stream=0)
    assert _call(coli, _norm(coli, gate=1), d=None, r=None, g=None, ro=None, y=None, T=0) == 0


def test_binding_refuses_tensors_it_would_misread(coli):
    import torch
    w = torch.ones(64)
    with pytest.raises(ValueError):
        coli.BlockNorm(32, pre_w=w)
    with pytest.raises(TypeError):
        coli.BlockNorm(64, post_w=w.bfloat16())
    with pytest.raises(KeyError):
        coli.BlockNorm(64, gate="head")
    n = coli.BlockNorm(64, pre_w=w, gate="token")
    x = torch.zeros(3, 64)
    ok = dict(residual=x, block_out=x.clone(), residual_out=x.clone(), normed_out=x.clone(), gate=torch.zeros(3), stream=0)

    def call(**over):
        kw = dict(ok, **over)
        coli.residual_norm(n, kw["residual"], kw["block_out"], kw["residual_out"], kw["normed_out"], gate=kw["gate"],
                           stream=kw["stream"])
    for over, err in ((dict(block_out=x[:2]), ValueError), (dict(residual_out=x.bfloat16()), TypeError),
                      (dict(normed_out=x.bfloat16()), TypeError), (dict(gate=torch.zeros(64)), ValueError),
                      (dict(gate=torch.zeros(3).bfloat16()), TypeError), (dict(residual=x.double()), TypeError),
                      (dict(block_out=torch.zeros(64, 3).t()), ValueError)):
        with pytest.raises(err):
            call(**over)
    with pytest.raises(ValueError):
        coli.residual_norm(coli.BlockNorm(64, pre_w=w), x, x.clone(), x.clone(), x.clone(), gate=torch.zeros(3), stream=0)
