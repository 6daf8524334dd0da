"""The bounded waits of the router's and the adapters' batch kernels, made to run
out on purpose (GPU): coli_debug_set_wait_ns shortens the limit so that the
pipeline waits give up.  A waiting thread looks at the clock each time the
barrier wakes it, so a wait that is over by then still succeeds: the call must
return and complete, its status word must be 1 or its result right, and the next
call with the normal limit must be right again.  A timed-out wait only stops
waiting: no fault, trap or endless wait is involved.
"""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    import torch
    import int4_routed_expert_bias_b200 as coli
    torch.cuda.init()
    yield coli, torch
    coli.debug_set_wait_ns(0)


def word(ws, torch):
    torch.cuda.synchronize()
    return int(ws[:4].view(torch.int32).item())


def times_out(coli, torch, call, ws):
    coli.debug_set_wait_ns(1)
    try:
        call()                    # returns normally
        status = word(ws, torch)  # and the launches complete
    finally:
        coli.debug_set_wait_ns(0)
    return status


@pytest.mark.parametrize("bf16", [True, False])
def test_router(env, bf16):
    coli, torch = env
    torch.manual_seed(0)
    T, H, E, k = 700, 4096, 160, 6
    x = torch.randn(T, H, device="cuda")
    x = x.bfloat16() if bf16 else x
    r = coli.Router(H, E, k, torch.randn(E, H, device="cuda") * H ** -0.5, n_group=8, topk_group=3)
    ws = torch.zeros(coli.router_workspace_size(r, T), dtype=torch.uint8, device="cuda")
    idx, w = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
    coli.router_forward(r, x, idx, w, ws)
    assert word(ws, torch) == 0
    want = idx.clone(), w.clone()
    status = times_out(coli, torch, lambda: coli.router_forward(r, x, idx, w, ws), ws)
    assert status == 1 or (status == 0 and torch.equal(idx, want[0]) and torch.equal(w, want[1]))
    assert bool(((idx >= 0) & (idx < E)).all())
    coli.router_forward(r, x, idx, w, ws)
    assert word(ws, torch) == 0
    assert torch.equal(idx, want[0]) and torch.equal(w, want[1])


@pytest.mark.parametrize("xt", ["bfloat16", "float32"])
def test_adapters(env, xt):
    coli, torch = env
    torch.manual_seed(1)
    T, K, N, R, n = 600, 4096, 2048, 64, 3
    dt = getattr(torch, xt)
    x, base = torch.randn(T, K, device="cuda").to(dt), torch.randn(T, N, device="cuda").to(dt)
    ad = coli.Adapters((torch.randn(n, R, K, device="cuda") * K ** -0.5).bfloat16(),
                       (torch.randn(n, N, R, device="cuda") * R ** -0.5).bfloat16(), torch.ones(n, device="cuda"))
    which = torch.randint(-1, n, (T,), device="cuda", dtype=torch.int32)
    out = torch.empty_like(base)
    ws = torch.zeros(coli.adapters_workspace_size(ad, T), dtype=torch.uint8, device="cuda")
    coli.adapters_forward(ad, x, which, out, ws, base=base)
    assert word(ws, torch) == 0
    want = out.clone()
    status = times_out(coli, torch, lambda: coli.adapters_forward(ad, x, which, out, ws, base=base), ws)
    assert status == 1 or (status == 0 and torch.equal(out, want))
    coli.adapters_forward(ad, x, which, out, ws, base=base)
    assert word(ws, torch) == 0
    assert torch.equal(out, want)
