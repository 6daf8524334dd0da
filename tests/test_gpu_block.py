"""The layer on a given routing, and the decoder block that runs the operators together (GPU).

With the layer's own routing handed back to it, every path has to give its own
output bit for bit.  Dropped slots and experts named twice are compared with
the routing that says the same in plain form, bit for bit, and with the formula
in 64 bits.  The block is compared with the single calls in its order, bit for
bit, and with the formulas in 64 bits end to end: the layer's own tolerances
(tests/_support.py: 2e-3 with fp32 accumulation, 1e-2 on the tensor cores, of a
token's largest output) reach the residual scaled by the block's factors, with
one bf16 rounding of the layer's output in between.
"""
import numpy as np
import pytest

import inputs
import _support as S

pytestmark = pytest.mark.gpu

SHAPES = [(1024, 512, 64, 8, 1, "single"), (1024, 512, 64, 8, 3, "decode"), (1024, 512, 64, 8, 33, "decode"),
          (256, 256, 300, 4, 40, "decode"), (256, 256, 16, 4, 100, "prefill"), (256, 256, 16, 4, 700, "prefill"),
          (256, 128, 16, 4, 130, "wide")]


@pytest.fixture(scope="module")
def env():
    import torch
    import int4_routed_expert_bias_b200 as coli
    torch.cuda.set_device(0)
    return coli, torch


def make(env, H, F, E, k, T, seed=0):
    coli, torch = env
    rng = np.random.default_rng(seed + H + 3 * T)
    ex = {}
    for e in range(E + 1):
        ex[e] = {}
        for name, N, K in (("gate", F, H), ("up", F, H), ("down", H, F)):
            q, s = inputs.quantise_gs64(rng.standard_normal((N, K)) * 0.03)
            ex[e][name + "_q"], ex[e][name + "_s"] = q, s
    stacked = inputs.stack_experts(ex, E)
    c = inputs.Config(0, "given", H, F, E, k, T, "f32", "f32", 1)
    w_router = (rng.standard_normal((E, H)) * 0.05).astype(np.float32)
    sel_bias = (rng.standard_normal(E) * 0.02).astype(np.float32)
    L = S.upload_layer(coli, torch, c, w_router, sel_bias, stacked)
    return L, {n: a for n, a in stacked.items()}, rng


def ffn64(st, e, x):
    """Expert e on rows x in double, from the stored nibbles and scales."""
    def w(name):
        b = np.asarray(st[name + "_q"][e]).view(np.uint8)
        q = np.stack([b & 15, b >> 4], axis=-1).reshape(b.shape[0], -1).astype(np.int64)
        q = np.where(q > 7, q - 16, q)
        return q * np.repeat(np.asarray(st[name + "_s"][e], np.float64), 64, axis=1)
    g, u = x @ w("gate").T, x @ w("up").T
    return (g / (1 + np.exp(-g)) * u) @ w("down").T


def layer64(st, E, x, idx, w):
    out = ffn64(st, E, x)
    for e in range(E):
        t, j = np.nonzero(idx == e)
        rows = np.unique(t)
        if len(rows):
            y = ffn64(st, e, x[rows])
            for i, r in enumerate(rows):
                out[r] += w[r][idx[r] == e].sum() * y[i]
    return out


def routed(env, L, x, idx, w, ot=None):
    coli, torch = env
    T = x.shape[0]
    out = torch.full((T + 1, L.hidden), 7.0, device="cuda", dtype=ot or x.dtype)
    ws = torch.full((coli.moe_workspace_size(L, T),), 0xEE, dtype=torch.uint8, device="cuda")
    coli.moe_forward_routed(L, x, idx, w, out[:T], ws)
    torch.cuda.synchronize()
    off = coli.moe_status_word_offset(L, T)
    assert int(ws[off:off + 4].view(torch.int32)[0]) == 0
    assert bool((out[T] == 7).all())
    return out[:T]


@pytest.mark.parametrize("H,F,E,k,T,path", SHAPES)
@pytest.mark.parametrize("bf16", [False, True])
def test_own_routing_handed_back(env, H, F, E, k, T, path, bf16):
    coli, torch = env
    L, st, rng = make(env, H, F, E, k, T)
    assert coli.moe_path(L, T) == path
    x = torch.from_numpy(rng.standard_normal((T, H)).astype(np.float32)).cuda()
    x = x.bfloat16() if bf16 else x
    out, idx = torch.empty_like(x), torch.empty(T, k, dtype=torch.int32, device="cuda")
    w = torch.empty(T, k, device="cuda")
    ws = torch.empty(coli.moe_workspace_size(L, T), dtype=torch.uint8, device="cuda")
    coli.moe_forward(L, x, out, ws, idx, w)
    assert torch.equal(routed(env, L, x, idx, w), out)


@pytest.mark.parametrize("H,F,E,k,T,path", SHAPES)
def test_dropped_and_repeated_experts(env, H, F, E, k, T, path):
    coli, torch = env
    L, st, rng = make(env, H, F, E, k, T, seed=5)
    x = torch.from_numpy(rng.standard_normal((T, H)).astype(np.float32)).cuda()
    idx = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    w = rng.standard_normal((T, k)).astype(np.float32)
    plain_i, plain_w = idx.copy(), w.copy()
    for t in range(T):
        kind = t % 4
        if kind == 0:          # the same expert in slots 0 and k - 1
            idx[t, k - 1] = plain_i[t, 0]
            idx[t, 0] = plain_i[t, 0]
            plain_w[t, 0] = w[t, 0] + w[t, k - 1]
            plain_i[t, k - 1], plain_w[t, k - 1] = -1, 0
        elif kind == 1:        # out of range both ways
            idx[t, 0], idx[t, 1] = E, -2 ** 31
            plain_i[t, :2], plain_w[t, :2] = -1, 0
        elif kind == 2 and t % 8 == 2:  # nothing but the shared expert
            idx[t], plain_i[t], plain_w[t] = 2 ** 31 - 1, -1, 0
    def dev(a):
        return torch.from_numpy(np.ascontiguousarray(a)).cuda()
    got = routed(env, L, x, dev(idx), dev(w))
    assert torch.equal(got, routed(env, L, x, dev(plain_i), dev(plain_w)))
    want = layer64(st, E, x.double().cpu().numpy(), plain_i, plain_w.astype(np.float64))
    S.check_output(got.cpu().numpy(), want, S.TOL_PREFILL if path == "prefill" else S.TOL_DECODE, path)


def test_routed_call_in_a_graph(env):
    coli, torch = env
    for H, F, E, k, T, path in SHAPES:
        L, st, rng = make(env, H, F, E, k, T, seed=6)
        x = torch.from_numpy(rng.standard_normal((T, H)).astype(np.float32)).cuda()
        idx = torch.from_numpy(np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)).cuda()
        w = torch.rand(T, k, device="cuda")
        want = routed(env, L, x, idx, w)
        iin, win, out = torch.zeros_like(idx), torch.zeros_like(w), torch.empty_like(x)
        ws = torch.empty(coli.moe_workspace_size(L, T), dtype=torch.uint8, device="cuda")
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            coli.moe_forward_routed(L, x, iin, win, out, ws)
        iin.copy_(idx)
        win.copy_(w)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def block_parts(env, H, F, E, k, T, own_router, adapters, seed=0):
    coli, torch = env
    L, st, rng = make(env, H, F, E, k, T, seed)

    def dev(a):
        return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).cuda()
    router = None
    if not own_router:
        router = coli.Router(H, E, k, dev(rng.standard_normal((E, H)) * 0.05), None, score="softmax", n_group=2, topk_group=1,
                             group_top=2, renormalise=True, routed_scale=1.7)
    before = coli.BlockNorm(H, pre_w=dev(1 + 0.1 * rng.standard_normal(H)), post_w=dev(1 + 0.1 * rng.standard_normal(H)))
    after = coli.BlockNorm(H, pre_w=dev(1 + 0.1 * rng.standard_normal(H)), post_w=dev(1 + 0.1 * rng.standard_normal(H)),
                           gate="token", gate_sigmoid=True, block_scale=0.5)
    ad = None
    if adapters:
        ad = coli.Adapters((dev(rng.standard_normal((3, 16, H))) * H ** -0.5).bfloat16(),
                           (dev(rng.standard_normal((3, H, 16))) * 0.02).bfloat16(), torch.ones(3, device="cuda"))
    return coli.Block(L, before, after, router=router, adapters=ad), st, rng


@pytest.mark.parametrize("H,F,E,k,T,path", SHAPES)
@pytest.mark.parametrize("own_router", [False, True])
@pytest.mark.parametrize("adapters", [False, True])
def test_block_is_its_calls(env, H, F, E, k, T, path, own_router, adapters):
    coli, torch = env
    blk, st, rng = block_parts(env, H, F, E, k, T, own_router, adapters)
    prev = torch.from_numpy(rng.standard_normal((T, H)).astype(np.float32)).cuda().bfloat16()
    r = torch.from_numpy(2 * rng.standard_normal((T, H)).astype(np.float32)).cuda()
    gate = torch.from_numpy(rng.standard_normal(T).astype(np.float32)).cuda().bfloat16()
    which = torch.from_numpy(rng.integers(-1, 3, T).astype(np.int32)).cuda() if adapters else None
    # the calls, one by one
    r1, x = torch.empty_like(r), torch.empty_like(prev)
    coli.residual_norm(blk.norm_before, r, prev, r1, x)
    y = torch.empty_like(x)
    lws = torch.empty(coli.moe_workspace_size(blk.layer, T), dtype=torch.uint8, device="cuda")
    idx, w = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
    if own_router:
        coli.moe_forward(blk.layer, x, y, lws, idx, w)
    else:
        rws = torch.empty(coli.router_workspace_size(blk.router, T), dtype=torch.uint8, device="cuda")
        coli.router_forward(blk.router, x, idx, w, rws)
        coli.moe_forward_routed(blk.layer, x, idx, w, y, lws)
    y_layer = y.clone()
    if adapters:
        aws = torch.empty(coli.adapters_workspace_size(blk.adapters, T), dtype=torch.uint8, device="cuda")
        coli.adapters_forward(blk.adapters, x, which, y, aws, base=y)
    r2, nxt = torch.empty_like(r), torch.empty_like(x)
    coli.residual_norm(blk.norm_after, r1, y, r2, nxt, gate=gate)
    # the block
    ws = torch.full((coli.moe_block_workspace_size(blk, torch.bfloat16, T),), 0xEE, dtype=torch.uint8, device="cuda")
    ro, no = torch.empty_like(r), torch.empty_like(x)
    coli.moe_block_forward(blk, r, prev, ro, no, ws, which=which, gate_after=gate)
    torch.cuda.synchronize()
    assert torch.equal(ro, r2) and torch.equal(no, nxt)
    for off in coli.moe_block_status_word_offsets(blk, torch.bfloat16, T):
        assert off is None or int(ws[off:off + 4].view(torch.int32)[0]) == 0
    # in place, and replayed from a graph
    rin, nin = r.clone(), torch.empty_like(x)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        coli.moe_block_forward(blk, rin, prev, rin, nin, ws, which=which, gate_after=gate)
    rin.copy_(r)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(rin, r2) and torch.equal(nin, nxt)
    # end to end in double, from the routing taken (the router's own test holds it to double)
    want = layer64(st, E, x.double().cpu().numpy(), idx.cpu().numpy(), w.double().cpu().numpy())
    tol = S.TOL_PREFILL if path == "prefill" else S.TOL_DECODE
    S.check_output(y_layer.float().cpu().numpy(), want, tol + 2.0 ** -8, path)
    if adapters:
        for i in range(3):
            rows = np.nonzero(which.cpu().numpy() == i)[0]
            a, b = (t[i].double().cpu().numpy() for t in (blk.adapters.tensors["a"], blk.adapters.tensors["b"]))
            want[rows] += x.double().cpu().numpy()[rows] @ a.T @ b.T
    pw = blk.norm_after.tensors["post_w"].double().cpu().numpy()
    d = want / np.sqrt((want ** 2).mean(axis=1, keepdims=True) + 1e-5) * pw
    d = d * (0.5 / (1 + np.exp(-gate.double().cpu().numpy())))[:, None]
    res = r1.double().cpu().numpy() + d
    # a relative error e of the layer's largest output is at most 2 e of the normalised row's largest value
    # (its own and its norm's); one bf16 rounding each of y and, with adapters, of their sum
    bound = 2 * (tol + 2 * 2.0 ** -8) * np.abs(d).max(axis=1, keepdims=True) * np.abs(pw).max() / np.abs(pw).min() + 1e-6 * np.abs(res)
    assert (np.abs(ro.double().cpu().numpy() - res) <= bound).all()


def test_first_block_and_last_block(env):
    """No previous output (the residual alone is normalised); no norm of the next input."""
    coli, torch = env
    H, F, E, k, T = 256, 256, 16, 4, 9
    L, st, rng = make(env, H, F, E, k, T)
    w = torch.ones(H, device="cuda")
    blk = coli.Block(L, coli.BlockNorm(H, pre_w=w), coli.BlockNorm(H))
    r = torch.from_numpy(rng.standard_normal((T, H)).astype(np.float32)).cuda()
    ro = torch.empty_like(r)
    ws = torch.empty(coli.moe_block_workspace_size(blk, torch.float32, T), dtype=torch.uint8, device="cuda")
    coli.moe_block_forward(blk, r, None, ro, None, ws)
    x, y = torch.empty_like(r), torch.empty_like(r)
    coli.residual_norm(blk.norm_before, r, None, None, x)
    lws = torch.empty(coli.moe_workspace_size(L, T), dtype=torch.uint8, device="cuda")
    coli.moe_forward(L, x, y, lws)
    torch.cuda.synchronize()
    assert torch.equal(ro, r + y)
