"""The residual norm (coli_residual_norm) against its formulas in 64 bits.

Tolerance.  With u = 2^-24: a mean of squares is summed in fp32 by threads of at
most 16 values and a tree of 10, relative error at most 32 u, so its reciprocal
root carries 16 u + 4 u; the factors and the weights add at most 8 roundings.
So a block term f d is within 28 u of itself, r' within 30 u (|rs r| + |bs f d|),
and y within q w times that plus another 28 u |y| for its own mean, whose value
moves by the errors of r': 30 u of the row's root mean square of |rs r| + |bs f d|.
Each output is then rounded once to its type: eps / 2 of its value.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module")
def env():
    import torch
    import int4_routed_expert_bias_b200 as coli
    torch.cuda.set_device(0)
    return coli, torch


def f64(t):
    return t.double().cpu().numpy()


def check(env, T, H, xt="bf16", rt="bf16", post=True, pre=True, gate="none", sigmoid=False, rs=1.0, bs=1.0, block=True,
          in_place=False, scale=1.0, seed=0, eps=1e-5, with_residual=True):
    coli, torch = env
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 31 * T + H)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")
    d = (normal(T, H) * scale).to(dt[xt]) if block else None
    r = (normal(T, H) * 3 * scale).to(dt[rt])
    post_w = normal(H) if post else None
    pre_w = normal(H) if pre else None
    gt = {"none": None, "channel": (H,), "token": (T,), "element": (T, H)}[gate]
    gt = None if gt is None else normal(*gt).to(dt[xt])
    norm = coli.BlockNorm(H, post_w=post_w, pre_w=pre_w, eps=eps, gate=gate, gate_sigmoid=sigmoid, residual_scale=rs,
                          block_scale=bs)
    # the reference
    r64 = rs * f64(r)
    mag = np.abs(r64)
    new = r64
    if block:
        d64 = f64(d)
        if post:
            d64 = d64 / np.sqrt((d64 ** 2).mean(axis=1, keepdims=True) + eps) * f64(post_w)
        if gate != "none":
            g64 = f64(gt)
            g64 = 1 / (1 + np.exp(-g64)) if sigmoid else g64
            d64 = d64 * (g64[:, None] if gate == "token" else g64)
        new = r64 + bs * d64
        mag = mag + np.abs(bs * d64)
    # outputs with a guard row behind them
    ro = torch.full((T + 1, H), 7.0, device="cuda", dtype=r.dtype)
    y = torch.full((T + 1, H), 7.0, device="cuda", dtype=dt[xt])
    if in_place:
        ro[:T] = r
        r = ro[:T]
        if block:
            y[:T] = d
            d = y[:T]
    coli.residual_norm(norm, r, d, ro[:T] if with_residual else None, y[:T] if pre else None, gate=gt)
    torch.cuda.synchronize()
    if with_residual:
        assert bool((ro[T] == 7).all())
        err = np.abs(f64(ro[:T]) - new)
        tol = 30 * U * mag + torch.finfo(ro.dtype).eps / 2 * (np.abs(new) + 30 * U * mag)
        assert (err <= tol).all(), float((err / tol).max())
    if pre:
        assert bool((y[T] == 7).all())
        q = 1 / np.sqrt((new ** 2).mean(axis=1, keepdims=True) + eps)
        w = np.abs(f64(pre_w))
        y64 = new * q * f64(pre_w)
        moved = 30 * U * np.sqrt((mag ** 2).mean(axis=1, keepdims=True)) * q
        tol = 30 * U * mag * q * w + (28 * U + moved) * np.abs(y64)
        tol = tol + torch.finfo(y.dtype).eps / 2 * (np.abs(y64) + tol)
        err = np.abs(f64(y[:T]) - y64)
        assert (err <= tol).all(), float((err / tol).max())
    return ro, y


@pytest.mark.parametrize("xt,rt", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("T,H", [(1, 1), (3, 7), (2, 8), (5, 120), (9, 128), (4, 129), (17, 256), (3, 264), (8, 512), (2, 520),
                                 (1, 1021), (33, 1024), (2, 4096), (3, 4100), (3, 4097), (1, 6144), (150, 2048), (2, 16384),
                                 (1, 16383)])
def test_widths(env, T, H, xt, rt):
    check(env, T, H, xt, rt)


@pytest.mark.parametrize("T,H", [(2049, 4096), (1200, 7000), (8200, 1032), (1025, 8192)])
@pytest.mark.parametrize("xt,rt", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32"), ("f32", "bf16")])
def test_long_batches(env, T, H, xt, rt):
    """Batches whose rows are walked (no norm of the block's output), and the same with it."""
    check(env, T, H, xt, rt, post=False, gate="channel", in_place=True)
    check(env, T, H, xt, rt, post=False, pre=False, gate="element", sigmoid=True)
    check(env, T, H, xt, rt, post=False, block=False, with_residual=False)
    check(env, T, H, xt, rt, post=True)


@pytest.mark.parametrize("H", [192, 77, 1536, 6000])
@pytest.mark.parametrize("gate", ["none", "channel", "token", "element"])
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("post,pre", [(True, True), (True, False), (False, True), (False, False)])
def test_forms(env, H, gate, sigmoid, post, pre):
    check(env, 6, H, "bf16", "f32", post, pre, gate, sigmoid, rs=0.9, bs=-0.5)
    check(env, 6, H, "f32", "f32", post, pre, gate, sigmoid, rs=1.5, bs=0.25, in_place=True)


@pytest.mark.parametrize("H", [64, 1000, 2048])
def test_without_a_block(env, H):
    """The first block's input: only the residual is there, and it may stay unwritten."""
    check(env, 5, H, "bf16", "bf16", post=False, block=False)
    check(env, 5, H, "bf16", "f32", post=False, block=False, with_residual=False)


def test_largest_batch(env):
    """65536 x 16384 (2^30 values, 2 GB a tensor): rows from all over."""
    coli, torch = env
    T, H = 65536, 16384
    g = torch.Generator(device="cuda")
    g.manual_seed(0)
    d, r = (torch.empty(T, H, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    for i in range(0, T, 8192):
        d[i:i + 8192] = torch.randn(8192, H, generator=g, device="cuda")
        r[i:i + 8192] = torch.randn(8192, H, generator=g, device="cuda") * 2
    w = torch.randn(H, generator=g, device="cuda")
    rows = torch.tensor([0, 1, 32767, 32768, 40001, 65535], device="cuda")
    new = f64(r[rows]) + f64(d[rows])
    y = new / np.sqrt((new ** 2).mean(axis=1, keepdims=True) + 1e-5) * f64(w)
    coli.residual_norm(coli.BlockNorm(H, pre_w=w), r, d, r, d)  # in place
    torch.cuda.synchronize()
    assert (np.abs(f64(r[rows]) - new) <= 2.0 ** -8 * np.abs(new) + 1e-5).all()
    assert (np.abs(f64(d[rows]) - y) <= 2.0 ** -8 * np.abs(y) + 1e-4).all()


@pytest.mark.parametrize("scale", [1e-18, 1e-6, 1e6, 1e17])
def test_magnitudes(env, scale):
    check(env, 4, 1024, "f32", "f32", scale=scale, eps=0.0)
    check(env, 4, 1024, "bf16", "f32", scale=scale, eps=1e-5 * min(1.0, scale) ** 2)


def test_rows_do_not_touch_each_other(env):
    """A row of NaN and one of zeros: only the NaN row is NaN, zeros stay finite (eps)."""
    coli, torch = env
    for H in (256, 1536):
        r, d = torch.randn(6, H, device="cuda"), torch.randn(6, H, device="cuda")
        r[2] = float("nan")
        r[4] = 0
        d[4] = 0
        w = torch.randn(H, device="cuda")
        ro, y = torch.empty_like(r), torch.empty_like(d)
        coli.residual_norm(coli.BlockNorm(H, post_w=w, pre_w=w), r, d, ro, y)
        nan = torch.isnan(y).any(dim=1).tolist()
        assert nan == [False, False, True, False, False, False]
        assert bool((y[4] == 0).all()) and bool((ro[4] == 0).all())


def test_streams_and_graphs(env):
    coli, torch = env
    H, T = 2048, 70
    w = torch.randn(H, device="cuda")
    n = coli.BlockNorm(H, post_w=w, pre_w=w)
    r, d = torch.randn(T, H, device="cuda"), torch.randn(T, H, device="cuda").bfloat16()
    want_r, want_y = torch.empty_like(r), torch.empty_like(d)
    coli.residual_norm(n, r, d, want_r, want_y)
    ro, y = torch.empty_like(r), torch.empty_like(d)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    coli.residual_norm(n, r, d, ro, y, stream=side)
    side.synchronize()
    assert torch.equal(ro, want_r) and torch.equal(y, want_y)
    g = torch.cuda.CUDAGraph()
    rin = torch.zeros_like(r)
    with torch.cuda.graph(g):
        coli.residual_norm(n, rin, d, ro, y)
    rin.copy_(r)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(ro, want_r) and torch.equal(y, want_y)
