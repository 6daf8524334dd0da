"""Host-only checks of the adapters' arguments (no GPU, nothing launched)."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def coli():
    from int4_routed_expert_bias_b200 import _build
    _build.build()
    import int4_routed_expert_bias_b200 as m
    return m


X, WH, BASE, OUT, WS, A, B, S, RK = ((i + 1) << 32 for i in range(9))  # far apart, aligned, never read


def _ad(coli, **over):
    kw = dict(in_features=1024, out_features=512, max_rank=16, n_adapters=4, a=A, b=B, scale=S, rank=RK)
    kw.update(over)
    s = coli._AdaptersStruct()
    for k, v in kw.items():
        setattr(s, k, v)
    return s


def _call(coli, d, x=X, xt=1, T=4, which=WH, base=BASE, out=OUT, ot=1, ws=WS, n=1 << 40):
    return coli.lib().coli_adapters_forward(ctypes.byref(d) if d is not None else None, x, xt, T, which, base, out, ot, ws, n,
                                            None)


@pytest.mark.parametrize("over", [
    dict(in_features=0), dict(in_features=1020), dict(in_features=65544), dict(out_features=4), dict(out_features=508),
    dict(out_features=65544), dict(max_rank=0), dict(max_rank=12), dict(max_rank=264), dict(n_adapters=0),
    dict(n_adapters=1025), dict(a=None), dict(b=None), dict(scale=None), dict(a=A + 8), dict(b=B + 2), dict(scale=S + 2),
    dict(rank=RK + 1)])
def test_bad_adapters_are_refused(coli, over):
    d = _ad(coli, **over)
    assert _call(coli, d) == 1
    assert coli.last_error()
    assert coli.lib().coli_adapters_workspace_size(ctypes.byref(d), 1) == 0


@pytest.mark.parametrize("over", [
    dict(xt=2), dict(ot=-1), dict(T=-1), dict(T=65537), dict(x=None), dict(which=None), dict(out=None), dict(ws=None),
    dict(x=X + 8), dict(base=BASE + 4), dict(out=OUT + 2), dict(which=WH + 1), dict(ws=WS + 16), dict(out=X),
    dict(out=X + 4 * 1024 * 2 - 16), dict(out=BASE + 16), dict(base=OUT - 1024)])
def test_bad_call_is_refused(coli, over):
    assert _call(coli, _ad(coli), **over) == 1
    assert coli.last_error()


def test_short_workspace_null_and_empty(coli):
    d = _ad(coli, rank=None)
    need = coli.lib().coli_adapters_workspace_size(ctypes.byref(d), 100)
    assert need > 0
    assert _call(coli, d, T=100, n=need - 1) == 3
    assert _call(coli, None) == 1
    assert _call(coli, d, T=0, x=None, which=None, base=None, out=None, ws=None, n=0) == 0
    assert coli.lib().coli_adapters_workspace_size(ctypes.byref(d), 0) > 0


def test_binding_refuses_tensors_it_would_misread(coli):
    import torch
    a, b, s = torch.zeros(3, 8, 64).bfloat16(), torch.zeros(3, 32, 8).bfloat16(), torch.ones(3)
    with pytest.raises(TypeError):
        coli.Adapters(a.float(), b, s)
    with pytest.raises(ValueError):
        coli.Adapters(a, b[:2], s)
    with pytest.raises(ValueError):
        coli.Adapters(a, b, s[:2])
    with pytest.raises(TypeError):
        coli.Adapters(a, b, s, rank=torch.ones(3, dtype=torch.int64))
    d = coli.Adapters(a, b, s)
    x, which, out, ws = torch.zeros(5, 64), torch.zeros(5, dtype=torch.int32), torch.zeros(5, 32), torch.zeros(1 << 16).byte()
    for args, err in (((x[:, :56], which, out, ws), ValueError), ((x, which.long(), out, ws), TypeError),
                      ((x, which[:4], out, ws), ValueError), ((x, which, out.half(), ws), TypeError)):
        with pytest.raises(err):
            coli.adapters_forward(d, *args, stream=0)
    with pytest.raises(TypeError):
        coli.adapters_forward(d, x, which, out, ws, base=out.bfloat16(), stream=0)
    with pytest.raises(coli.ColiError):
        coli.adapters_workspace_size(d, -1)
