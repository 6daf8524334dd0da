"""Host-only checks of the given-routing call and of the decoder block (no GPU, nothing launched)."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def coli():
    from int4_routed_expert_bias_b200 import _build
    _build.build()
    import int4_routed_expert_bias_b200 as m
    return m


def at(i):
    return (i + 1) << 36  # far apart, aligned, never read


def _layer(coli, **over):
    kw = dict(hidden=1024, ffn=512, n_experts=64, top_k=4, group=64, routed_scale=2.5, w_router=at(0), sel_bias=at(0),
              gate_q=at(0), up_q=at(0), down_q=at(0), gate_s=at(0), up_s=at(0), down_s=at(0))
    kw.update(over)
    s = coli._LayerStruct()
    for k, v in kw.items():
        setattr(s, k, v)
    return s


def _routed(coli, L, x=at(1), xt=1, T=2, idx=at(2), w=at(3), out=at(4), ot=1, ws=at(5), n=1 << 40):
    return coli.lib().coli_moe_forward_routed(ctypes.byref(L), x, xt, T, idx, w, out, ot, ws, n, None)


@pytest.mark.parametrize("over", [dict(x=None), dict(idx=None), dict(w=None), dict(out=None), dict(ws=None), dict(idx=at(2) + 2),
                                  dict(w=at(3) + 1), dict(x=at(1) + 8), dict(T=-1), dict(xt=3), dict(ot=3), dict(ws=at(5) + 8)])
def test_bad_routed_call_is_refused(coli, over):
    assert _routed(coli, _layer(coli), **over) == 1
    assert coli.last_error()


def test_routed_call_of_a_layer_without_a_router(coli):
    L = _layer(coli, w_router=None, sel_bias=None)
    size = coli.lib().coli_moe_workspace_size(ctypes.byref(L), 2)
    assert size > 0
    assert _routed(coli, L, n=size - 1) == 3
    assert _routed(coli, L, T=0, x=None, idx=None, w=None, out=None, ws=None) == 0
    # its own routing is not there to be used, and half a router is none
    assert coli.lib().coli_moe_forward(ctypes.byref(L), at(1), 1, 2, at(4), 1, at(5), 1 << 40, None, None, None) == 1
    assert _routed(coli, _layer(coli, w_router=None)) == 1
    assert _routed(coli, _layer(coli, sel_bias=None)) == 1
    assert _routed(coli, _layer(coli, act_int8=1), T=65) == 2


class _Parts:
    def __init__(self, coli, **over):
        kw = dict(layer=_layer(coli), router=coli._RouterStruct(1024, 64, 4, 0, 1, 1, 1, 1, 1.0, at(0), None),
                  before=coli._BlockNormStruct(1024, 1e-5, at(0), at(0), 0, 0, 1.0, 1.0),
                  after=coli._BlockNormStruct(1024, 1e-5, at(0), at(0), 2, 1, 1.0, 1.0),
                  adapters=coli._AdaptersStruct(1024, 1024, 16, 4, at(0), at(0), at(0), None))
        kw.update(over)
        self.parts = kw
        a = {k: None if v is None else ctypes.addressof(v) for k, v in kw.items()}
        self.block = coli._BlockStruct(a["layer"], a["router"], a["before"], a["after"], a["adapters"])


def _block(coli, b, prev=at(1), xt=1, r=at(2), rt=0, g0=None, g1=at(3), which=at(4), T=3, ro=at(5), nx=at(6), ws=at(7), n=1 << 40):
    return coli.lib().coli_moe_block_forward(ctypes.byref(b.block), prev, xt, r, rt, g0, g1, which, T, ro, nx, ws, n, None)


@pytest.mark.parametrize("over", [
    dict(xt=2), dict(rt=2), dict(T=-1), dict(T=65537), dict(r=None), dict(ro=None), dict(nx=None), dict(prev=None),
    dict(g1=None), dict(which=None), dict(which=at(4) + 2), dict(ws=None), dict(ws=at(7) + 16), dict(ro=at(1)),
    dict(nx=at(5)), dict(nx=at(5) + 64), dict(prev=at(1) + 2)])
def test_bad_block_call_is_refused(coli, over):
    b = _Parts(coli)
    assert _block(coli, b, **over) == 1
    assert coli.last_error()


def test_block_parts_must_fit(coli):
    size = coli.lib().coli_moe_block_workspace_size
    good = _Parts(coli)
    need = size(ctypes.byref(good.block), 1, 3)
    assert need > 0 and _block(coli, good, n=need - 1) == 3
    for over in (dict(layer=None), dict(before=None), dict(after=None),
                 dict(before=coli._BlockNormStruct(1024, 1e-5, None, None, 0, 0, 1.0, 1.0)),
                 dict(before=coli._BlockNormStruct(512, 1e-5, None, at(0), 0, 0, 1.0, 1.0)),
                 dict(after=coli._BlockNormStruct(512, 1e-5, None, at(0), 0, 0, 1.0, 1.0)),
                 dict(router=coli._RouterStruct(1024, 32, 4, 0, 1, 1, 1, 1, 1.0, at(0), None)),
                 dict(router=coli._RouterStruct(1024, 64, 5, 0, 1, 1, 1, 1, 1.0, at(0), None)),
                 dict(router=coli._RouterStruct(1024, 64, 4, 0, 7, 1, 1, 1, 1.0, at(0), None)),
                 dict(router=None, layer=_layer(coli, w_router=None, sel_bias=None)),
                 dict(adapters=coli._AdaptersStruct(1024, 512, 16, 4, at(0), at(0), at(0), None)),
                 dict(adapters=coli._AdaptersStruct(1024, 1024, 12, 4, at(0), at(0), at(0), None)),
                 dict(layer=_layer(coli, hidden=960))):
        b = _Parts(coli, **over)
        assert size(ctypes.byref(b.block), 1, 3) == 0
        assert _block(coli, b) == 1
    assert size(ctypes.byref(good.block), 2, 3) == 0
    assert _block(coli, good, T=0, prev=None, r=None, ro=None, nx=None, ws=None, n=0) == 0


def test_block_status_words(coli):
    b = _Parts(coli)
    r, l = ctypes.c_size_t(), ctypes.c_size_t()
    f = coli.lib().coli_moe_block_status_word_offsets
    for T in (1, 100):
        assert f(ctypes.byref(b.block), 1, T, ctypes.byref(r), ctypes.byref(l)) == 0
        size = coli.lib().coli_moe_block_workspace_size(ctypes.byref(b.block), 1, T)
        assert r.value % 256 == 0 and l.value % 4 == 0 and r.value != l.value and max(r.value, l.value) + 4 <= size
    none = ctypes.c_size_t(-1).value
    b = _Parts(coli, router=None)
    assert f(ctypes.byref(b.block), 1, 4, ctypes.byref(r), ctypes.byref(l)) == 0 and r.value == none
    assert f(ctypes.byref(b.block), 1, 4, None, ctypes.byref(l)) == 1


def test_empty_tensors(coli):
    """A batch of no tokens: tensors without elements have no address, and nothing needs one."""
    import torch
    H, F, E, k = 64, 64, 8, 2
    w = torch.randn(E, H)
    x, idx, wt = torch.empty(0, H), torch.empty(0, k, dtype=torch.int32), torch.empty(0, k)
    which, ws = torch.empty(0, dtype=torch.int32), torch.empty(0, dtype=torch.uint8)
    out = [torch.empty(0, H) for _ in range(3)]

    def experts(n, m):
        return torch.zeros(E + 1, n, m // 2, dtype=torch.uint8), torch.zeros(E + 1, n, m // 64)

    router = coli.Router(H, E, k, w)
    adapters = coli.Adapters(torch.zeros(2, 8, H).bfloat16(), torch.zeros(2, H, 8).bfloat16(), torch.ones(2))
    layer = coli.Layer(H, F, E, k, 1.0, w, torch.zeros(E), *experts(F, H), *experts(F, H), *experts(H, F))
    norm = coli.BlockNorm(H, pre_w=torch.ones(H))
    block = coli.Block(layer, norm, norm, router=router, adapters=adapters)
    coli.router_forward(router, x, idx, wt, ws, stream=0)
    coli.adapters_forward(adapters, x, which, out[0], ws, base=out[1], stream=0)
    coli.moe_forward_routed(layer, x, idx, wt, out[0], ws, stream=0)
    coli.residual_norm(norm, x, out[0], out[1], out[2], stream=0)
    coli.moe_block_forward(block, x, out[0], out[1], out[2], ws, which=which, stream=0)
