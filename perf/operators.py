"""What the operators around the routed-expert layer are measured on.

Three operators, each in its plain form (elementary torch operations) and as the
library's call:

  router    Scores of a token against every expert (sigmoid or softmax of fp32
            weights times the token), a selection bias, groups of experts of
            which only the best are eligible, the k best experts in order and
            their weights.
  norm      The residual path around a block: the block's output normalised,
            gated and scaled into the residual, and the new residual normalised
            as the next block's input.
  adapters  Low-rank adapters of many requests in one batch, added beside a
            projection that all requests share.

`listed()` are the cases that stand for the range, `draw(rng)` makes more of the
same range.
"""
import numpy as np
import torch

own = False

# The decoder block that the sizes come from: hidden 6144, 256 routed experts,
# 8 per token, batches of 1 (decoding), 4 (a verify batch), 64 (a decode batch)
# and 4096 tokens (prefill).


def _router(name, T, H, E, k, x, score, groups, keep, top, bias, renorm, scale):
    return dict(name=name, op="router", T=T, H=H, E=E, k=k, x=x, score=score, groups=groups, keep=keep, top=top,
                bias=bias, renorm=renorm, scale=scale)


def _norm(name, T, H, x, r, post, pre, gate, sigmoid, rscale, bscale):
    return dict(name=name, op="norm", T=T, H=H, x=x, r=r, post=post, pre=pre, gate=gate, sigmoid=sigmoid,
                rscale=rscale, bscale=bscale)


def _adapters(name, T, K, N, R, n, x, ragged, sorted_, none):
    return dict(name=name, op="adapters", T=T, K=K, N=N, R=R, n=n, x=x, ragged=ragged, sorted=sorted_, none=none)


def listed():
    return [
        # one token being decoded: the router of the layer, with experts in eight groups of which four are eligible
        _router("router-decode-1", 1, 6144, 256, 8, "bf16", "sigmoid", 8, 4, 2, True, True, 2.5),
        # a decode batch of 64 requests on a smaller softmax router without groups
        _router("router-decode-64", 64, 2048, 64, 6, "bf16", "softmax", 1, 1, 1, False, False, 1.0),
        # a ragged batch of fp32 activations, softmax scores, groups ranked by their best expert
        _router("router-ragged-1003", 1003, 5120, 160, 6, "f32", "softmax", 8, 3, 1, False, True, 16.0),
        # prefill of 4096 tokens on the layer's router
        _router("router-prefill-4096", 4096, 6144, 256, 8, "bf16", "sigmoid", 8, 4, 2, True, True, 2.5),
        # one token: the block's output normalised and gated into the residual, and the next block's input
        _norm("norm-decode-1", 1, 6144, "bf16", "bf16", True, True, "token", True, 1.0, 1.0),
        # an odd width and an odd batch in fp32, a gate for every element
        _norm("norm-odd-333", 333, 1021, "f32", "f32", True, True, "element", False, 1.0, 0.5),
        # prefill of 4096 tokens: residual add and the norm before the block
        _norm("norm-prefill-4096", 4096, 6144, "bf16", "bf16", False, True, "none", False, 1.0, 1.0),
        # four such batches at once, an fp32 residual, a learned gate per channel, norms before and after
        _norm("norm-prefill-16384", 16384, 6144, "bf16", "f32", True, True, "channel", False, 1.0, 0.7),
        # a verify batch: four tokens of up to eight adapters of rank 16
        _adapters("adapters-verify-4", 4, 6144, 6144, 16, 8, "bf16", False, False, False),
        # a decode batch of 64 requests over 32 adapters of ranks up to 64, some requests without one
        _adapters("adapters-decode-64", 64, 6144, 2048, 64, 32, "bf16", True, False, True),
        # a ragged fp32 batch in no order
        _adapters("adapters-ragged-1003", 1003, 2048, 6144, 24, 7, "f32", True, False, True),
        # prefill of 4096 tokens of several requests, each request's tokens in a row
        _adapters("adapters-prefill-4096", 4096, 6144, 6144, 64, 16, "bf16", False, True, False),
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], spread evenly over its logarithm."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["router", "norm", "adapters"])
    if op == "router":
        groups = rng.choice([1, 1, 2, 4, 8])
        per = rng.randint(4, 64 if groups <= 4 else 32)
        E = groups * per
        keep = rng.randint(1, groups)
        k = rng.randint(1, min(16, keep * per))
        H = 8 * _log(rng, 64, 1024)
        T = _log(rng, 1, min(4096, 4096 * 6144 * 256 // (H * max(E, 256))))
        return _router("", T, H, E, k, rng.choice(["bf16", "bf16", "f32"]), rng.choice(["sigmoid", "softmax"]), groups,
                       keep, rng.choice([1, 2]), rng.random() < 0.5, rng.random() < 0.7, rng.choice([1.0, 2.5, 16.0]))
    if op == "norm":
        H = _log(rng, 64, 8192)
        if rng.random() < 0.7:
            H = max(64, H // 64 * 64)
        T = _log(rng, 1, min(16384, 16384 * 6144 // H))
        post = rng.random() < 0.5
        return _norm("", T, H, rng.choice(["bf16", "bf16", "f32"]), rng.choice(["bf16", "f32"]), post,
                     not post or rng.random() < 0.7, rng.choice(["none", "channel", "token", "element"]),
                     rng.random() < 0.5, rng.choice([1.0, 0.9]), rng.choice([1.0, 0.5]))
    K, N = 8 * _log(rng, 32, 1024), 8 * _log(rng, 32, 1024)
    R = rng.choice([8, 16, 24, 32, 64, 128])
    n = _log(rng, 1, 64)
    T = _log(rng, 1, min(4096, max(1, 4096 * 1024 * 12288 // (R * n * (K + N)))))
    return _adapters("", T, K, N, R, n, rng.choice(["bf16", "bf16", "f32"]), rng.random() < 0.5, rng.random() < 0.5,
                     rng.random() < 0.5)


_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_SIZE = {"bf16": 2, "f32": 4}


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, std=1.0, dt=torch.float32):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(dt)

    s = dict(case)
    T = case["T"]
    if case["op"] == "router":
        H, E, k = case["H"], case["E"], case["k"]
        # normalised activations; a few channels are much larger, as in trained models
        x = normal(T, H)
        x[:, torch.randint(0, H, (4,), generator=g, device="cuda")] *= 8.0
        s["x_"] = x.to(_DT[case["x"]])
        s["w_router"] = normal(E, H, std=1.5 / H ** 0.5)
        s["sel_bias"] = normal(E, std=0.05) if case["bias"] else None
        s["idx_out"] = torch.empty(T, k, dtype=torch.int32, device="cuda")
        s["w_out"] = torch.empty(T, k, dtype=torch.float32, device="cuda")
        if own:
            import int4_routed_expert_bias_b200 as coli
            s["handle"] = coli.Router(H, E, k, s["w_router"], s["sel_bias"], score=case["score"],
                                      n_group=case["groups"], topk_group=case["keep"], group_top=case["top"],
                                      renormalise=case["renorm"], routed_scale=case["scale"])
            s["ws"] = torch.empty(coli.router_workspace_size(s["handle"], T), dtype=torch.uint8, device="cuda")
    elif case["op"] == "norm":
        H = case["H"]
        s["block_out"] = normal(T, H, std=0.7, dt=_DT[case["x"]])
        s["residual"] = normal(T, H, std=3.0, dt=_DT[case["r"]])
        s["post_w"] = normal(H, std=0.2) + 1.0 if case["post"] else None
        s["pre_w"] = normal(H, std=0.2) + 1.0 if case["pre"] else None
        s["gate_"] = {"none": lambda: None, "channel": lambda: normal(H, dt=_DT[case["x"]]),
                      "token": lambda: normal(T, dt=_DT[case["x"]]),
                      "element": lambda: normal(T, H, dt=_DT[case["x"]])}[case["gate"]]()
        s["residual_out"] = torch.empty_like(s["residual"])
        s["normed_out"] = torch.empty_like(s["block_out"]) if case["pre"] else None
        if own:
            import int4_routed_expert_bias_b200 as coli
            s["handle"] = coli.BlockNorm(H, post_w=s["post_w"], pre_w=s["pre_w"], eps=1e-5, gate=case["gate"],
                                         gate_sigmoid=case["sigmoid"], residual_scale=case["rscale"],
                                         block_scale=case["bscale"])
    else:
        K, N, R, n = case["K"], case["N"], case["R"], case["n"]
        s["x_"] = normal(T, K, dt=_DT[case["x"]])
        s["base"] = normal(T, N, dt=_DT[case["x"]])
        s["a"] = normal(n, R, K, std=K ** -0.5, dt=torch.bfloat16)
        s["b"] = normal(n, N, R, std=R ** -0.5, dt=torch.bfloat16)
        s["scale"] = torch.rand(n, generator=g, device="cuda") * 1.5 + 0.5
        s["rank"] = (torch.randint(1, R + 1, (n,), generator=g, device="cuda", dtype=torch.int32)
                     if case["ragged"] else None)
        which = torch.randint(-1 if case["none"] else 0, n, (T,), generator=g, device="cuda", dtype=torch.int32)
        s["which"] = torch.sort(which).values if case["sorted"] else which
        s["out"] = torch.empty_like(s["base"])
        if own:
            import int4_routed_expert_bias_b200 as coli
            s["handle"] = coli.Adapters(s["a"], s["b"], s["scale"], rank=s["rank"])
            s["ws"] = torch.empty(coli.adapters_workspace_size(s["handle"], T), dtype=torch.uint8, device="cuda")
    return s


# --- plain forms ---------------------------------------------------------------------------------------------


def _plain_router(s):
    """In 64 bits: which of two experts comes first is decided by their scores' last bits."""
    T, E, G = s["T"], s["E"], s["groups"]
    z = s["x_"].double() @ s["w_router"].double().T
    if s["score"] == "sigmoid":
        p = 1.0 / (1.0 + torch.exp(-z))
    else:
        e = torch.exp(z - z.max(dim=1, keepdim=True).values)
        p = e / e.sum(dim=1, keepdim=True)
    c = p if s["sel_bias"] is None else p + s["sel_bias"].double()
    if G > 1:
        per = c.view(T, G, E // G)
        best = torch.sort(per, dim=2, descending=True).values[:, :, :s["top"]].sum(dim=2)
        kept = torch.sort(best, dim=1, descending=True, stable=True).indices[:, :s["keep"]]
        on = torch.zeros(T, G, dtype=torch.bool, device=c.device)
        on[torch.arange(T, device=c.device)[:, None], kept] = True
        c = torch.where(on[:, :, None], per, torch.full_like(per, -float("inf"))).view(T, E)
    idx = torch.sort(c, dim=1, descending=True, stable=True).indices[:, :s["k"]]
    w = torch.gather(p, 1, idx)
    if s["renorm"]:
        w = w / w.sum(dim=1, keepdim=True)
    return {"idx": idx.int(), "w": (w * s["scale"]).float()}


def _plain_norm(s):
    d, r = s["block_out"].float(), s["residual"].float()
    if s["post_w"] is not None:
        d = d * torch.rsqrt((d * d).mean(dim=1, keepdim=True) + 1e-5) * s["post_w"]
    if s["gate_"] is not None:
        gate = s["gate_"].float()
        if s["sigmoid"]:
            gate = 1.0 / (1.0 + torch.exp(-gate))
        d = d * (gate[:, None] if s["gate"] == "token" else gate)
    r = r * s["rscale"] + d * s["bscale"]
    out = {"residual": r.to(s["residual"].dtype)}
    if s["pre_w"] is not None:
        y = r * torch.rsqrt((r * r).mean(dim=1, keepdim=True) + 1e-5) * s["pre_w"]
        out["normed"] = y.to(s["block_out"].dtype)
    return out


def _plain_adapters(s):
    T, K, N, R, n = s["T"], s["K"], s["N"], s["R"], s["n"]
    h = (s["x_"].float() @ s["a"].float().view(n * R, K).T).view(T, n, R)
    on = (s["which"][:, None] == torch.arange(n, device=h.device))[:, :, None]
    if s["rank"] is not None:
        on = on & (torch.arange(R, device=h.device) < s["rank"][:, None])
    h = torch.where(on, h * s["scale"][:, None], torch.zeros_like(h))
    y = s["base"].float() + h.view(T, n * R) @ s["b"].float().permute(0, 2, 1).reshape(n * R, N)
    return {"out": y.to(s["base"].dtype)}


def run(state):
    s = state
    if own:
        import int4_routed_expert_bias_b200 as coli
        if s["op"] == "router":
            coli.router_forward(s["handle"], s["x_"], s["idx_out"], s["w_out"], s["ws"])
            return {"idx": s["idx_out"], "w": s["w_out"]}
        if s["op"] == "norm":
            coli.residual_norm(s["handle"], s["residual"], s["block_out"], s["residual_out"], s["normed_out"],
                               gate=s["gate_"])
            out = {"residual": s["residual_out"]}
            if s["normed_out"] is not None:
                out["normed"] = s["normed_out"]
            return out
        coli.adapters_forward(s["handle"], s["x_"], s["which"], s["out"], s["ws"], base=s["base"])
        return {"out": s["out"]}
    return {"router": _plain_router, "norm": _plain_norm, "adapters": _plain_adapters}[s["op"]](s)


def work(case):
    T = case["T"]
    if case["op"] == "router":
        H, E, k = case["H"], case["E"], case["k"]
        return {"bytes": T * H * _SIZE[case["x"]] + E * H * 4 + (E * 4 if case["bias"] else 0) + T * k * 8,
                "flops": 2 * T * H * E}
    if case["op"] == "norm":
        H, x, r = case["H"], _SIZE[case["x"]], _SIZE[case["r"]]
        gate = {"none": 0, "channel": H, "token": T, "element": T * H}[case["gate"]] * x
        weights = (case["post"] + case["pre"]) * H * 4
        return {"bytes": T * H * (x + 2 * r + (x if case["pre"] else 0)) + gate + weights,
                "flops": T * H * (3 + 4 * case["post"] + 4 * case["pre"] + (case["gate"] != "none"))}
    K, N, R, n, x = case["K"], case["N"], case["R"], case["n"], _SIZE[case["x"]]
    # the adapters that the batch can touch, their mean rank, the tokens that have one
    rank = (R + 1) / 2 if case["ragged"] else R
    tokens = T * n / (n + 1) if case["none"] else T
    used = n * (1.0 - (1.0 - 1.0 / (n + case["none"])) ** T)
    return {"bytes": int(tokens * K * x + 2 * T * N * x + used * rank * (K + N) * 2 + T * 4),
            "flops": int(2 * tokens * rank * (K + N))}


# --- from the definitions, in 64 bits on the host --------------------------------------------------------------


def _host(t):
    return None if t is None else t.detach().cpu().to(torch.float64).numpy()


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "router":
        x, W, bias = _host(s["x_"]), _host(s["w_router"]), _host(s["sel_bias"])
        T, E, G, k = case["T"], case["E"], case["groups"], case["k"]
        z = x @ W.T
        if case["score"] == "sigmoid":
            p = np.where(z >= 0, 1 / (1 + np.exp(-np.abs(z))), np.exp(-np.abs(z)) / (1 + np.exp(-np.abs(z))))
        else:
            p = np.exp(z - np.logaddexp.reduce(z, axis=1, keepdims=True))
        c = p + (0 if bias is None else bias)
        idx, w = np.zeros((T, k), np.int32), np.zeros((T, k))
        for t in range(T):
            allowed = range(E)
            if G > 1:
                m = E // G
                value = [sum(sorted(c[t, i * m:(i + 1) * m], reverse=True)[:case["top"]]) for i in range(G)]
                groups = sorted(range(G), key=lambda i: (-value[i], i))[:case["keep"]]
                allowed = [e for i in sorted(groups) for e in range(i * m, (i + 1) * m)]
            idx[t] = sorted(allowed, key=lambda e: (-c[t, e], e))[:k]
            w[t] = p[t, idx[t]]
        if case["renorm"]:
            w /= w.sum(axis=1, keepdims=True)
        return {"idx": idx, "w": w * case["scale"]}
    if case["op"] == "norm":
        def rms(v):
            return v / np.sqrt(np.einsum("th,th->t", v, v)[:, None] / v.shape[1] + 1e-5)

        d = _host(s["block_out"])
        if case["post"]:
            d = rms(d) * _host(s["post_w"])
        if case["gate"] != "none":
            gate = _host(s["gate_"])
            gate = 1 / (1 + np.exp(-gate)) if case["sigmoid"] else gate
            d = d * (gate.reshape(-1, 1) if case["gate"] == "token" else gate)
        r = case["rscale"] * _host(s["residual"]) + case["bscale"] * d
        out = {"residual": r}
        if case["pre"]:
            out["normed"] = rms(r) * _host(s["pre_w"])
        return out
    x, a, b, scale = _host(s["x_"]), _host(s["a"]), _host(s["b"]), _host(s["scale"])
    which, out = s["which"].cpu().numpy(), _host(s["base"])
    for i in range(case["n"]):
        rows = np.nonzero(which == i)[0]
        r = case["R"] if s["rank"] is None else int(s["rank"][i])
        if len(rows):
            out[rows] += scale[i] * (x[rows] @ a[i, :r].T) @ b[i, :, :r].T
    return {"out": out}
