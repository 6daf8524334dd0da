"""The general router (coli_router_forward) against its definition in 64 bits.

Indices have to be those of 64-bit arithmetic, near ties included, for one
token and for batches.  Tolerance of the weights: a score z is an fp32 sum of H
products; its error is taken as at most 8 roundings of the largest partial sum,
8 * 2^-24 * max|z| (the sums run in many short pieces), and sigmoid or softmax
move their value by at most twice that relatively; the exponential, the
quotients and the sum over k <= 32 slots add less than 48 roundings.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    import torch
    import int4_routed_expert_bias_b200 as coli
    torch.cuda.set_device(0)
    return coli, torch


def reference(x, W, bias, k, score, n_group, topk_group, group_top, renorm, scale):
    """The definition, in double on the host; x and W are float64 arrays of the stored values."""
    z = x @ W.T
    T, E = z.shape
    if score == "sigmoid":
        s = 1 / (1 + np.exp(-z))
    else:
        s = np.exp(z - z.max(axis=1, keepdims=True))
        s /= s.sum(axis=1, keepdims=True)
    c = s + (0 if bias is None else bias)
    m = E // n_group
    idx = np.zeros((T, k), np.int64)
    for t in range(T):
        best = [np.sort(c[t, g * m:(g + 1) * m])[::-1][:group_top].sum() for g in range(n_group)]
        groups = set(sorted(range(n_group), key=lambda g: (-best[g], g))[:topk_group])
        idx[t] = sorted((e for e in range(E) if e // m in groups), key=lambda e: (-c[t, e], e))[:k]
    w = np.take_along_axis(s, idx, 1)
    if renorm:
        w = w / w.sum(axis=1, keepdims=True)
    return idx, w * scale, np.abs(z).max(axis=1)


def route(env, x, W, bias, k, **kw):
    coli, torch = env
    r = coli.Router(W.shape[1], W.shape[0], k, W, bias, **kw)
    T = x.shape[0]
    ws = torch.full((coli.router_workspace_size(r, T) + 64,), 0xA5, dtype=torch.uint8, device="cuda")
    idx = torch.full((T + 1, k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T + 1, k), -7.0, device="cuda")
    coli.router_forward(r, x, idx[:T], w[:T], ws[:-64])
    torch.cuda.synchronize()
    assert int(ws[:4].view(torch.int32)[0]) == 0
    # rows behind the last token and bytes behind the workspace stay as they were
    assert bool((idx[T] == -7).all()) and bool((w[T] == -7).all()) and bool((ws[-64:] == 0xA5).all())
    return idx[:T], w[:T]


def check(env, x, W, bias, k, score="sigmoid", n_group=1, topk_group=1, group_top=2, renormalise=True, routed_scale=1.0):
    idx, w = route(env, x, W, bias, k, score=score, n_group=n_group, topk_group=topk_group, group_top=group_top,
                   renormalise=renormalise, routed_scale=routed_scale)
    ridx, rw, zmax = reference(x.double().cpu().numpy(), W.double().cpu().numpy(),
                               None if bias is None else bias.double().cpu().numpy(), k, score, n_group, topk_group,
                               group_top if n_group > 1 else 1, renormalise, routed_scale)
    assert np.array_equal(idx.cpu().numpy(), ridx)
    tol = 2 ** -24 * (2 * 2 * 8 * zmax[:, None] + 48)
    err = np.abs(w.double().cpu().numpy() - rw) / np.abs(rw)
    assert (err <= tol).all(), float((err / tol).max())


def inputs(torch, T, H, E, bf16, seed, std=1.5):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = torch.randn(T, H, generator=g, device="cuda")
    W = torch.randn(E, H, generator=g, device="cuda") * (std / H ** 0.5)
    b = torch.randn(E, generator=g, device="cuda") * 0.05
    return (x.bfloat16() if bf16 else x), W, b


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("T", [1, 2, 3, 7, 8, 9, 33, 129, 300])
def test_batches_of_the_layers_router(env, T, bf16):
    x, W, b = inputs(env[1], T, 1024, 256, bf16, T)
    check(env, x, W, b, 8, n_group=8, topk_group=4, routed_scale=2.5)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("H,E,k,G,keep,top,bias,renorm", [
    (8, 1, 1, 1, 1, 1, False, True),        # one expert
    (8, 2, 2, 1, 1, 1, True, False),        # every expert selected
    (72, 7, 3, 1, 1, 1, True, True),        # odd expert count, H not a multiple of 64
    (520, 33, 32, 1, 1, 1, True, True),     # the largest k
    (136, 96, 5, 32, 3, 1, True, False),    # the most groups, three experts each
    (264, 60, 4, 3, 2, 2, False, True),     # group count not a power of two
    (1000, 160, 6, 8, 3, 1, True, False),
    (2056, 1024, 16, 4, 1, 2, True, True),  # the most experts
    (16384, 130, 8, 1, 1, 1, False, True),  # the widest row
    (64, 512, 9, 16, 16, 2, True, True),    # every group kept
    (512, 16, 4, 8, 2, 2, True, True),      # the k experts are all of the kept groups
])
@pytest.mark.parametrize("T", [1, 5, 70])
def test_shapes(env, T, H, E, k, G, keep, top, bias, renorm, score):
    x, W, b = inputs(env[1], T, H, E, T % 2 == 1, H + E + T)
    check(env, x, W, b if bias else None, k, score=score, n_group=G, topk_group=keep, group_top=top, renormalise=renorm,
          routed_scale=0.75)


@pytest.mark.parametrize("E", [31, 100, 127, 200, 284, 290, 513, 700, 1000])
def test_long_batches_of_any_expert_count(env, E):
    """The selection kernel packs as many tokens into a block as its shared memory holds."""
    x, W, b = inputs(env[1], 2400, 64, E, True, E)
    check(env, x, W, b, 5)


@pytest.mark.parametrize("bf16,H", [(True, 16384), (False, 9000)])
def test_largest_batch(env, bf16, H):
    """65536 tokens (the inputs pass 2^31 bytes): rows from all over against the definition."""
    coli, torch = env
    T, E, k = 65536, 24, 4
    x, W, b = inputs(torch, T, H, E, bf16, 3)
    idx, w = route(env, x, W, b, k, n_group=4, topk_group=2)
    rows = torch.tensor([0, 1, 255, 256, 32767, 32768, 40000, 65279, 65534, 65535], device="cuda")
    ridx, rw, _ = reference(x[rows].double().cpu().numpy(), W.double().cpu().numpy(), b.double().cpu().numpy(), k, "sigmoid",
                            4, 2, 2, True, 1.0)
    assert np.array_equal(idx[rows].cpu().numpy(), ridx)
    assert np.abs(w[rows].double().cpu().numpy() - rw).max() < 1e-5


@pytest.mark.parametrize("T", [1, 4, 40, 200])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("bias", [False, True])
def test_near_ties_are_decided_as_in_double(env, T, score, bias):
    """Experts in near-equal families: gaps of 1e-9 to 1e-5 between neighbours in
    rank, which fp32 sums cannot tell apart; equal rows go to the lower index."""
    coli, torch = env
    g = torch.Generator(device="cuda")
    g.manual_seed(T)
    H, E = 768, 64
    x = torch.randn(T, H, generator=g, device="cuda")
    W = torch.randn(8, H, generator=g, device="cuda").repeat(8, 1) * (1.5 / H ** 0.5)
    step = 10.0 ** -torch.arange(2, 10, device="cuda").float().repeat_interleave(8)
    W = W * (1 + step[:, None] * torch.rand(E, 1, generator=g, device="cuda"))
    W[40:48] = W[0:8]  # exact ties
    b = (torch.arange(E, device="cuda") % 8).float() * 0.01 if bias else None
    check(env, x, W, b, 12, score=score)
    check(env, x, W, b, 6, score=score, n_group=8, topk_group=3, group_top=2)
    check(env, x, W, b, 6, score=score, n_group=8, topk_group=3, group_top=1)


def test_rows_of_zeros_and_masked_experts(env):
    """A padding row of zeros ties every expert (the bias or the index decides); a
    bias of -inf takes experts out of the choice."""
    coli, torch = env
    x, W, b = inputs(torch, 37, 512, 64, True, 5)
    x[::3] = 0
    check(env, x, W, b, 4, n_group=8, topk_group=2)
    check(env, x, W, None, 4, score="softmax")
    b[:] = -float("inf")
    b[[3, 17, 18, 40, 63]] = 0.0
    idx, w = route(env, x, W, b, 4)
    assert set(np.unique(idx.cpu().numpy())) <= {3, 17, 18, 40, 63}


@pytest.mark.parametrize("T", [1, 6, 90])
def test_tokens_that_are_not_finite(env, T):
    """NaN or infinite activations give k distinct experts for that token and leave the others alone."""
    coli, torch = env
    x, W, b = inputs(torch, T, 256, 48, False, 9)
    clean, cw = route(env, x, W, b, 5, n_group=4, topk_group=2)
    bad = list(range(0, T, 3))
    x[bad[0::2], 3] = float("nan")
    x[bad[1::2], 7] = float("inf")
    idx, w = route(env, x, W, b, 5, n_group=4, topk_group=2)
    i = idx.cpu().numpy()
    assert (i >= 0).all() and (i < 48).all() and all(len(set(r)) == 5 for r in i)
    good = [t for t in range(T) if t not in bad]
    assert torch.equal(idx[good], clean[good]) and torch.equal(w[good], cw[good])


def test_a_token_routes_alike_alone_and_in_a_batch(env):
    coli, torch = env
    x, W, b = inputs(torch, 150, 1536, 128, True, 11)
    idx, w = route(env, x, W, b, 8, n_group=4, topk_group=2)
    for t in range(0, 150, 13):
        i1, w1 = route(env, x[t:t + 1], W, b, 8, n_group=4, topk_group=2)
        assert torch.equal(i1[0], idx[t])
        assert float((w1[0] - w[t]).abs().max()) < 1e-5


def test_streams_graphs_and_repeats(env):
    """Bit-equal on the default stream, on another one, and replayed from a graph with new inputs."""
    coli, torch = env
    for T in (1, 100):
        x, W, b = inputs(torch, T, 512, 64, True, 21)
        x2, _, _ = inputs(torch, T, 512, 64, True, 22)
        want, want2 = route(env, x, W, b, 6), route(env, x2, W, b, 6)
        r = coli.Router(512, 64, 6, W, b)
        ws = torch.empty(coli.router_workspace_size(r, T), dtype=torch.uint8, device="cuda")
        idx, w, xin = torch.empty_like(want[0]), torch.empty_like(want[1]), x.clone()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        coli.router_forward(r, xin, idx, w, ws, stream=side)
        side.synchronize()
        assert torch.equal(idx, want[0]) and torch.equal(w, want[1])
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            coli.router_forward(r, xin, idx, w, ws)
        for src, ref in ((x2, want2), (x, want)):
            xin.copy_(src)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(idx, ref[0]) and torch.equal(w, ref[1])


def test_calls_at_once_and_a_graph_with_copies_and_branches(env):
    """Two streams with a workspace each, many times over, and a captured graph that
    copies its inputs in and runs two calls on branches."""
    coli, torch = env
    cases = []
    for T, bf16 in ((300, True), (700, False), (3, True)):
        x, W, b = inputs(torch, T, 1024, 96, bf16, 31 + T)
        want = route(env, x, W, b, 6, n_group=8, topk_group=3)
        r = coli.Router(1024, 96, 6, W, b, n_group=8, topk_group=3)
        ws = torch.empty(coli.router_workspace_size(r, T), dtype=torch.uint8, device="cuda")
        cases.append((r, x, torch.empty_like(want[0]), torch.empty_like(want[1]), ws, want))
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(20):
        for st, (r, x, idx, w, ws, _) in zip(streams, cases):
            coli.router_forward(r, x, idx, w, ws, stream=st)
    torch.cuda.synchronize()
    for r, x, idx, w, ws, want in cases:
        assert torch.equal(idx, want[0]) and torch.equal(w, want[1])
        idx.zero_(), w.zero_()
    xin = [torch.zeros_like(c[1]) for c in cases]
    g, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(g):
        main = torch.cuda.current_stream()
        for buf, c in zip(xin, cases):
            buf.copy_(c[1])
        side.wait_stream(main)
        with torch.cuda.stream(side):
            coli.router_forward(cases[0][0], xin[0], cases[0][2], cases[0][3], cases[0][4])
        for i in (1, 2):
            coli.router_forward(cases[i][0], xin[i], cases[i][2], cases[i][3], cases[i][4])
        main.wait_stream(side)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    for r, x, idx, w, ws, want in cases:
        assert torch.equal(idx, want[0]) and torch.equal(w, want[1])
