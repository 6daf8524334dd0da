"""Low-rank adapters (coli_adapters_forward) against their formula in 64 bits.

Tolerance.  The products of both stages are exact in the tensor core; a sum
runs through at most n accumulations of 16 products each, and each may drop up
to 2^-23 of the sum of magnitudes so far, so h is within (K / 16 * 3 + 16) 2^-23
of Sum|x a| (three parts of fp32 x), plus the scale's rounding.  With bf16
outputs h enters the second stage within 2^-16 of itself.  The second sum adds
(R / 16 * 3 + 4) 2^-23 of Sum|h b|, the addition of base one rounding, and out
is rounded to its type: eps / 2.
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


def f64(t):
    return t.double().cpu().numpy()


def make(env, T, K, N, R, n, xt, ot, ragged=True, none=True, seed=0):
    torch = env[1]
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 7 * T + K + N)
    x = torch.randn(T, K, generator=g, device="cuda").to(dt[xt])
    a = (torch.randn(n, R, K, generator=g, device="cuda") * K ** -0.5).bfloat16()
    b = (torch.randn(n, N, R, generator=g, device="cuda") * R ** -0.5).bfloat16()
    scale = torch.randn(n, generator=g, device="cuda")
    rank = torch.randint(0, R + 1, (n,), generator=g, device="cuda", dtype=torch.int32) if ragged else None
    if ragged:  # what lies behind an adapter's rank must not matter
        for i in range(n):
            a[i, int(rank[i]):] = float("nan")
            b[i, :, int(rank[i]):] = float("inf")
    which = torch.randint(-1 if none else 0, n, (T,), generator=g, device="cuda", dtype=torch.int32)
    base = torch.randn(T, N, generator=g, device="cuda").to(dt[ot])
    return x, a, b, scale, rank, which, base


def reference(x, a, b, scale, rank, which, base):
    """(out, error bound) in double."""
    x, a, b, scale, w = f64(x), f64(a), f64(b), f64(scale), which.cpu().numpy()
    out16 = base.dtype != __import__("torch").float32
    out = f64(base).copy()
    K, R = a.shape[2], a.shape[1]
    err = np.abs(out) * 2.0 ** -24
    for i in range(a.shape[0]):
        rows = np.nonzero(w == i)[0]
        r = R if rank is None else int(rank[i])
        if not len(rows) or not r:
            continue
        ai, bi = a[i, :r], b[i, :, :r]
        h = x[rows] @ ai.T
        dh = (K / 16 * 3 + 16) * 2.0 ** -23 * (np.abs(x[rows]) @ np.abs(ai).T) + (2.0 ** -24 + (2.0 ** -16 if out16 else 0)) * np.abs(h)
        y = scale[i] * h @ bi.T
        mag = np.abs(scale[i]) * np.abs(h) @ np.abs(bi).T
        out[rows] += y
        err[rows] += np.abs(scale[i]) * dh @ np.abs(bi).T + (R / 16 * 3 + 4) * 2.0 ** -23 * mag + 2.0 ** -24 * np.abs(y)
    return out, err


def run(env, x, a, b, scale, rank, which, base, in_place=False, stream=None):
    coli, torch = env
    T = x.shape[0]
    ad = coli.Adapters(a, b, scale, rank=rank)
    ws = torch.full((coli.adapters_workspace_size(ad, T) + 64,), 0xFF, dtype=torch.uint8, device="cuda")
    out = torch.full((T + 1, b.shape[1]), 7.0, device="cuda", dtype=base.dtype)
    if in_place:
        out[:T] = base
        base = out[:T]
    coli.adapters_forward(ad, x, which, out[:T], ws[:-64], base=base, stream=stream)
    torch.cuda.synchronize()
    assert bool((out[T] == 7).all()) and bool((ws[-64:] == 0xFF).all())
    return out[:T]


def check(env, T, K, N, R, n, xt="bf16", ot="bf16", in_place=False, **kw):
    t = make(env, T, K, N, R, n, xt, ot, **kw)
    out = run(env, *t, in_place=in_place)
    want, err = reference(*t)
    tol = err + env[1].finfo(out.dtype).eps / 2 * (np.abs(want) + err)
    off = np.abs(f64(out) - want)
    assert (off <= tol).all(), float((off / tol).max())
    # rows without an adapter are base itself
    free = (t[5] < 0).cpu().numpy()
    assert np.array_equal(f64(out)[free], f64(t[6])[free])


@pytest.mark.parametrize("xt,ot", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("T,K,N,R,n", [
    (1, 8, 8, 8, 1), (2, 256, 264, 16, 3), (5, 1000, 40, 24, 2), (16, 264, 1032, 64, 2), (17, 512, 96, 72, 1),
    (33, 2048, 256, 8, 1), (64, 320, 520, 40, 64), (64, 128, 128, 16, 1), (65, 328, 256, 32, 3), (130, 96, 2056, 128, 5),
    (257, 1024, 72, 256, 2), (1000, 72, 136, 16, 1000), (2050, 64, 64, 8, 1), (100, 8, 8, 8, 1024)])
def test_shapes(env, T, K, N, R, n, xt, ot):
    check(env, T, K, N, R, n, xt, ot)


@pytest.mark.parametrize("R", [56, 136, 184, 192, 200, 248])
@pytest.mark.parametrize("ot", ["bf16", "f32"])
def test_high_ranks(env, R, ot):
    """What of the shared memory is left for base rows and B changes with the rank."""
    check(env, 150, 264, 456, R, 2, ot, ot, ragged=R % 3 == 0)
    check(env, 30, 264, 456, R, 2, ot, ot, ragged=R % 3 == 0)


def test_long_batch_grouping(env):
    """More tokens than the grouping keeps in registers."""
    check(env, 9001, 64, 72, 8, 5)
    check(env, 65536, 8, 8, 8, 1000, "f32", "f32")


@pytest.mark.parametrize("xt", ["bf16", "f32"])
def test_inputs_beyond_32_bit_offsets(env, xt):
    """x of 2.4e9 values: rows from all over against the formula."""
    coli, torch = env
    T, K, N, R, n = 36800, 65536, 16, 8, 3
    dt = torch.bfloat16 if xt == "bf16" else torch.float32
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    x = torch.empty(T, K, dtype=dt, device="cuda")
    for i in range(0, T, 4600):
        x[i:i + 4600] = torch.randn(min(4600, T - i), K, generator=g, device="cuda").to(dt)
    a = (torch.randn(n, R, K, generator=g, device="cuda") * K ** -0.5).bfloat16()
    b = torch.randn(n, N, R, generator=g, device="cuda").bfloat16()
    which = torch.randint(0, n, (T,), generator=g, device="cuda", dtype=torch.int32)
    ad = coli.Adapters(a, b, torch.ones(n, device="cuda"))
    ws = torch.empty(coli.adapters_workspace_size(ad, T), dtype=torch.uint8, device="cuda")
    out = torch.empty(T, N, device="cuda")
    coli.adapters_forward(ad, x, which, out, ws)
    rows = torch.tensor([0, 127, 128, 16383, 16384, 32767, 32768, 32769, 36799], device="cuda")
    want, err = reference(x[rows], a, b, torch.ones(n, device="cuda"), None, which[rows], torch.zeros(len(rows), N, device="cuda"))
    assert (np.abs(f64(out[rows]) - want) <= err * 1.0001).all()


@pytest.mark.parametrize("T", [3, 50, 64, 65, 300])
def test_in_place_and_full_rank(env, T):
    check(env, T, 512, 384, 32, 4, in_place=True)
    check(env, T, 512, 384, 32, 4, "f32", "f32", in_place=True, ragged=False, none=False)


@pytest.mark.parametrize("T", [1, 40, 200])
def test_without_base(env, T):
    coli, torch = env
    x, a, b, scale, rank, which, base = make(env, T, 256, 128, 16, 3, "bf16", "f32")
    ad = coli.Adapters(a, b, scale, rank=rank)
    ws = torch.empty(coli.adapters_workspace_size(ad, T), dtype=torch.uint8, device="cuda")
    out = torch.full((T, 128), float("nan"), device="cuda")
    coli.adapters_forward(ad, x, which, out, ws)
    want, err = reference(x, a, b, scale, rank, which, torch.zeros_like(base))
    assert (np.abs(f64(out) - want) <= err * 1.0001 + 1e-30).all()


@pytest.mark.parametrize("T", [5, 64, 500])
def test_no_token_has_an_adapter(env, T):
    """All outside [0, n): base comes back bit for bit, whatever the number is."""
    torch = env[1]
    x, a, b, scale, rank, which, base = make(env, T, 64, 72, 8, 2, "f32", "bf16")
    for w in (-1, 2, 2 ** 31 - 1, -2 ** 31):
        which.fill_(w)
        assert torch.equal(run(env, x, a, b, scale, rank, which, base), base)


@pytest.mark.parametrize("T", [60, 400])
def test_a_tokens_result_does_not_depend_on_its_company(env, T):
    """Permuted batches give permuted outputs bit for bit; a NaN row stays alone."""
    torch = env[1]
    x, a, b, scale, rank, which, base = make(env, T, 520, 200, 24, 6, "f32", "f32")
    out = run(env, x, a, b, scale, rank, which, base)
    p = torch.randperm(T, device="cuda")
    assert torch.equal(run(env, x[p], a, b, scale, rank, which[p], base[p]), out[p])
    x[3] = float("nan")
    which[3] = 0
    rank[0] = 5
    a[0, :5], b[0, :, :5] = 0.5, 0.5
    got = run(env, x, a, b, scale, rank, which, base)
    bad = torch.isnan(got).any(dim=1)
    assert bool(bad[3]) and int(bad.sum()) == 1


def test_streams_and_graphs(env):
    coli, torch = env
    for T in (20, 150):
        x, a, b, scale, rank, which, base = make(env, T, 512, 256, 16, 4, "bf16", "bf16")
        want = run(env, x, a, b, scale, rank, which, base)
        ad = coli.Adapters(a, b, scale, rank=rank)
        ws = torch.empty(coli.adapters_workspace_size(ad, T), dtype=torch.uint8, device="cuda")
        out = torch.empty_like(base)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        coli.adapters_forward(ad, x, which, out, ws, base=base, stream=side)
        side.synchronize()
        assert torch.equal(out, want)
        g = torch.cuda.CUDAGraph()
        xin, win = torch.zeros_like(x), torch.zeros_like(which)
        with torch.cuda.graph(g):
            coli.adapters_forward(ad, xin, win, out, ws, base=base)
        xin.copy_(x)
        win.copy_(which)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_calls_at_once_and_a_graph_with_copies_and_branches(env):
    """Streams with a workspace each, many times over, and a captured graph that
    copies its inputs in and runs calls on branches."""
    coli, torch = env
    cases = []
    for T, dt in ((20, "bf16"), (500, "f32"), (900, "bf16")):
        t = make(env, T, 512, 384, 32, 4, dt, dt)
        want = run(env, *t)
        ad = coli.Adapters(t[1], t[2], t[3], rank=t[4])
        ws = torch.empty(coli.adapters_workspace_size(ad, T), dtype=torch.uint8, device="cuda")
        cases.append((ad, t[0], t[5], t[6], torch.empty_like(t[6]), ws, want))
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(20):
        for st, (ad, x, which, base, out, ws, _) in zip(streams, cases):
            coli.adapters_forward(ad, x, which, out, ws, base=base, stream=st)
    torch.cuda.synchronize()
    for c in cases:
        assert torch.equal(c[4], c[6])
        c[4].zero_()
    xin = [torch.zeros_like(c[1]) for c in cases]
    g, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(g):
        main = torch.cuda.current_stream()
        for buf, c in zip(xin, cases):
            buf.copy_(c[1])
        side.wait_stream(main)
        with torch.cuda.stream(side):
            coli.adapters_forward(cases[0][0], xin[0], cases[0][2], cases[0][4], cases[0][5], base=cases[0][3])
            coli.adapters_forward(cases[1][0], xin[1], cases[1][2], cases[1][4], cases[1][5], base=cases[1][3])
        coli.adapters_forward(cases[2][0], xin[2], cases[2][2], cases[2][4], cases[2][5], base=cases[2][3])
        main.wait_stream(side)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    for c in cases:
        assert torch.equal(c[4], c[6])
