"""Host-only checks of the general router's arguments (no GPU, nothing launched)."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def coli():
    from int4_routed_expert_bias_b200 import _build
    _build.build()
    import int4_routed_expert_bias_b200 as m
    return m


FAKE = 1 << 20  # non-null and aligned: argument checks never read through it


def _router(coli, **over):
    kw = dict(hidden=1024, n_experts=64, top_k=4, score=0, n_group=8, topk_group=2, group_top=2, renormalise=1,
              routed_scale=1.0, w_router=FAKE, sel_bias=FAKE)
    kw.update(over)
    s = coli._RouterStruct()
    for k, v in kw.items():
        setattr(s, k, v)
    return s


def _call(coli, r, x=FAKE, xt=0, T=1, idx=FAKE, w=FAKE, ws=FAKE, n=1 << 40):
    return coli.lib().coli_router_forward(ctypes.byref(r) if r is not None else None, x, xt, T, idx, w, ws, n, None)


@pytest.mark.parametrize("over", [
    dict(hidden=0), dict(hidden=100), dict(hidden=16392), dict(n_experts=0), dict(n_experts=1032), dict(top_k=0),
    dict(top_k=33), dict(top_k=17), dict(score=2), dict(n_group=0), dict(n_group=7), dict(n_group=64), dict(topk_group=0),
    dict(topk_group=9), dict(group_top=0), dict(group_top=3), dict(n_experts=8, top_k=1), dict(renormalise=2),
    dict(routed_scale=float("nan")), dict(routed_scale=float("inf")), dict(w_router=None), dict(w_router=FAKE + 4),
    dict(sel_bias=FAKE + 2)])
def test_bad_router_is_refused(coli, over):
    r = _router(coli, **over)
    assert _call(coli, r) == 1
    assert coli.last_error()
    assert coli.lib().coli_router_workspace_size(ctypes.byref(r), 1) == 0


@pytest.mark.parametrize("over", [
    dict(x=None), dict(x=FAKE + 8), dict(xt=2), dict(T=-1), dict(T=65537), dict(idx=None), dict(w=None), dict(idx=FAKE + 2),
    dict(ws=None), dict(ws=FAKE + 16)])
def test_bad_call_is_refused(coli, over):
    assert _call(coli, _router(coli), **over) == 1
    assert coli.last_error()


def test_null_router_and_short_workspace(coli):
    assert _call(coli, None) == 1
    r = _router(coli)
    need = coli.lib().coli_router_workspace_size(ctypes.byref(r), 5)
    assert need > 0
    assert _call(coli, r, T=5, n=need - 1) == 3


def test_empty_batch_needs_nothing(coli):
    assert _call(coli, _router(coli), T=0, x=None, idx=None, w=None, ws=None, n=0) == 0


def test_workspace_grows_with_the_batch(coli):
    r = _router(coli, sel_bias=None)
    sizes = [coli.lib().coli_router_workspace_size(ctypes.byref(r), T) for T in (0, 1, 64, 4096, 65536)]
    assert all(s > 0 for s in sizes) and sizes[-1] > sizes[1]
    # every score of the largest batch has a place
    assert sizes[-1] >= 65536 * 64 * 4


def test_binding_refuses_tensors_it_would_misread(coli):
    import torch
    w = torch.zeros(64, 1024)
    with pytest.raises(ValueError):
        coli.Router(1024, 32, 4, w)
    with pytest.raises(TypeError):
        coli.Router(1024, 64, 4, w.double())
    with pytest.raises(ValueError):
        coli.Router(64, 1024, 4, w.t())
    with pytest.raises(ValueError):
        coli.Router(1024, 64, 4, w, sel_bias=torch.zeros(63))
    with pytest.raises(KeyError):
        coli.Router(1024, 64, 4, w, score="tanh")
    r = coli.Router(1024, 64, 4, w)
    ws = torch.zeros(1 << 20, dtype=torch.uint8)
    idx, wt = torch.zeros(2, 4, dtype=torch.int32), torch.zeros(2, 4)
    with pytest.raises(ValueError):
        coli.router_forward(r, torch.zeros(2, 1032), idx, wt, ws, stream=0)
    with pytest.raises(TypeError):
        coli.router_forward(r, torch.zeros(2, 1024).half(), idx, wt, ws, stream=0)
    with pytest.raises(TypeError):
        coli.router_forward(r, torch.zeros(2, 1024), idx.long(), wt, ws, stream=0)
    with pytest.raises(ValueError):
        coli.router_forward(r, torch.zeros(1024, 2).t(), idx, wt, ws, stream=0)
    with pytest.raises(coli.ColiError):
        coli.router_workspace_size(r, -1)
