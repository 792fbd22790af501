"""The operators measured: expert-grouped products with 16-bit weights and their
gradients, the weighted combine of expert rows and its gradient, and low-rank
adapters of many requests beside a shared projection and their gradients.

`run` takes one pass through an operator: as elementary torch operations in 32
bits, or (where `own` is set) as the package's calls. `exact` is the definition
in 64 bits. Sizes come from the layer shapes the package is built for (d = 2048,
f = 512, 256 experts, top-8; 16 experts, top-2) or are generic.
"""
import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # one decoded token, top-8 of 256 experts: gate/up rows of eight experts
        dict(name="experts_decode_1", op="gemm", tokens=1, top=8, groups=256, n=1024, k=2048, type="bf16", out="bf16", skew=0.0),
        # a short ragged batch over a few experts of odd widths (rows of no 16-byte alignment)
        dict(name="experts_odd", op="gemm", tokens=501, top=2, groups=13, n=515, k=777, type="fp16", out="fp32", skew=1.0),
        # a long prompt or training batch: gate/up product of the 256-expert layer
        dict(name="experts_train_8192", op="gemm", tokens=8192, top=8, groups=256, n=1024, k=2048, type="bf16", out="bf16", skew=0.5),
        # few wide experts, many rows each: bound by the matrix units
        dict(name="experts_few_wide", op="gemm", tokens=8192, top=2, groups=16, n=4096, k=2048, type="bf16", out="bf16", skew=0.2),
        # gradient of the gate/up product's input rows
        dict(name="experts_dgrad_4096", op="dgrad", tokens=4096, top=8, groups=256, n=1024, k=2048, type="bf16", out="bf16", skew=0.5),
        # gradient of the gate/up weights, added up in 32 bits by the trainer
        dict(name="experts_wgrad_8192", op="wgrad", tokens=8192, top=8, groups=64, n=1024, k=2048, type="bf16", out="fp32", skew=0.5),
        # the eight expert rows of each token of a long prompt, weighted and added
        dict(name="combine_8192", op="combine", tokens=8192, top=8, width=2048, type="bf16", out="bf16"),
        # its gradient: rows for the experts, weights for the router
        dict(name="combine_grad_2048", op="combine_grad", tokens=2048, top=8, width=2048, type="fp16", out="fp16"),
        # one decoded token with its request's adapter beside a projection
        dict(name="adapter_decode_1", op="adapter", tokens=1, adapters=8, n=2048, k=2048, rank=16, type="bf16", out="bf16", bare=0.0),
        # a decode batch: every request another adapter, some without one
        dict(name="adapter_decode_64", op="adapter", tokens=64, adapters=64, n=1024, k=2048, rank=16, type="fp16", out="fp16", bare=0.1),
        # prompts of 16 requests in one prefill batch
        dict(name="adapter_prefill_8192", op="adapter", tokens=8192, adapters=16, n=4096, k=2048, rank=32, type="bf16", out="bf16", bare=0.1),
        # training several adapters at once
        dict(name="adapter_grad_4096", op="adapter_grad", tokens=4096, adapters=4, n=2048, k=2048, rank=16, type="bf16", out="fp32", bare=0.0),
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def _width(rng, lo, hi):
    """A width of the range: mostly a multiple of 8 (rows of aligned vectors), else any."""
    w = _log(rng, lo, hi)
    return w if rng.random() < 0.2 else max(8, w // 8 * 8)


def draw(rng):
    op = rng.choice(["gemm", "gemm", "dgrad", "wgrad", "combine", "combine_grad", "adapter", "adapter", "adapter_grad"])
    t = rng.choice(["bf16", "fp16"])
    out = t if rng.random() < 0.6 else "fp32"
    if op in ("gemm", "dgrad", "wgrad"):
        top = rng.choice([1, 2, 4, 8])
        n, k = _width(rng, 64, 2048), _width(rng, 64, 2048)
        groups = max(top, _log(rng, 2, min(256, (1 << 28) // (n * k))))
        tokens = _log(rng, 1, min(65536, (1 << 37) // (n * k)) // top)
        return dict(op=op, tokens=tokens, top=top, groups=groups, n=n, k=k, type=t, out=out, skew=round(rng.random(), 2))
    if op in ("combine", "combine_grad"):
        top = rng.choice([1, 2, 4, 6, 8])
        return dict(op=op, tokens=_log(rng, 1, 65536 // top), top=top, width=_width(rng, 64, 2048), type=t, out=out if op == "combine" else t)
    return dict(op=op, tokens=_log(rng, 1, 8192), adapters=_log(rng, 1, 64), n=_width(rng, 64, 4096), k=_width(rng, 64, 2048),
                rank=rng.choice([4, 8, 16, 16, 32, 64, rng.randint(1, 64)]), type=t, out=out, bare=rng.choice([0.0, 0.1, 0.5]))


def _normal(g, shape, scale, dt):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dt)


def _route(g, tokens, top, groups, skew):
    """Expert choice as routing leaves it: (offsets, token of each sorted row, sorted row of each pair, longest group)."""
    score = torch.randn((tokens, groups), generator=g, device="cuda") + skew * torch.randn((groups,), generator=g, device="cuda")
    ids = torch.topk(score, top, dim=1).indices.reshape(-1)
    order = torch.sort(ids, stable=True).indices
    counts = torch.bincount(ids, minlength=groups)
    offsets = torch.zeros(groups + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = torch.cumsum(counts, 0).to(torch.int32)
    pos = torch.empty_like(order)
    pos[order] = torch.arange(order.numel(), device="cuda")
    return offsets, (order // top).to(torch.int32), pos.reshape(tokens, top).to(torch.int32), int(counts.max())


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt, op, T = _DT[case["type"]], case["op"], case["tokens"]
    s = dict(op=op, out=_DT[case["out"]])
    if op in ("gemm", "dgrad", "wgrad"):
        G, N, K = case["groups"], case["n"], case["k"]
        s["offsets"], s["token"], _, s["longest"] = _route(g, T, case["top"], G, case["skew"])
        P = T * case["top"]
        s["groups"] = G
        if op != "dgrad":
            s["x"] = _normal(g, (T, K), 1.0, dt)
        if op != "gemm":
            s["dc"] = _normal(g, (P, N), 1.0, dt)
        if op != "wgrad":
            s["w"] = _normal(g, (G, N, K), K ** -0.5, dt)
    elif op in ("combine", "combine_grad"):
        d, top = case["width"], case["top"]
        s["pos"] = _route(g, T, top, max(16, 2 * top), 0.5)[2]
        s["gate"] = torch.softmax(torch.randn((T, top), generator=g, device="cuda"), 1)
        s["o"] = _normal(g, (T * top, d), 1.0, dt)
        if op == "combine_grad":
            s["dy"] = _normal(g, (T, d), 1.0, dt)
        else:
            s["shared"] = _normal(g, (T, d), 1.0, dt)
    else:
        n, N, K, r = case["adapters"], case["n"], case["k"], case["rank"]
        ids = torch.randint(0, n, (T,), generator=g, device="cuda")
        # requests of a batch lie one after another; a decode batch has one row each
        ids = torch.sort(ids).values if T > 64 else ids
        ids = torch.where(torch.rand((T,), generator=g, device="cuda") < case["bare"], torch.full_like(ids, n), ids)
        s["order"] = torch.sort(ids, stable=True).indices.to(torch.int32)
        counts = torch.bincount(ids, minlength=n + 1)[:n]
        s["offsets"] = torch.zeros(n + 1, dtype=torch.int32, device="cuda")
        s["offsets"][1:] = torch.cumsum(counts, 0).to(torch.int32)
        s["longest"] = max(1, int(counts.max()))
        s["groups"] = n
        s["x"] = _normal(g, (T, K), 1.0, dt)
        s["a"] = _normal(g, (n, r, K), K ** -0.5, dt)
        s["b"] = _normal(g, (n, N, r), r ** -0.5, dt)
        s["scale"] = torch.rand((n,), generator=g, device="cuda") + 0.5
        if op == "adapter":
            s["base"] = _normal(g, (T, N), 1.0, s["out"])
        else:
            s["dy"] = _normal(g, (T, N), 1.0, dt)
            s["dx"] = _normal(g, (T, K), 1.0, dt)
    return s


# ------------------------------------------------------------------ plain form
def _places(offsets, rows):
    """Group and place in the group of each sorted row (group = number of groups for rows behind the last)."""
    p = torch.arange(rows, device=offsets.device, dtype=torch.int32)
    e = torch.searchsorted(offsets[1:].contiguous(), p, right=True)
    return e, p - offsets[e]


def _padded(x, e, at, groups, longest):
    """Rows laid out by group, each group filled up to the longest with zeros (the rows of no group go to an extra one)."""
    out = x.new_zeros((groups + 1, longest + 1, x.shape[1]))
    out[e, torch.clamp(at, max=longest)] = x
    return out[:groups, :longest]


def _plain_gemm(s):
    rows = s["token"].numel()
    e, at = _places(s["offsets"], rows)
    x = s["x"][s["token"]].float()
    if rows <= 64:  # few rows: each row with its own expert's weights
        return torch.matmul(s["w"][e].float(), x.unsqueeze(2)).squeeze(2).to(s["out"])
    c = torch.matmul(_padded(x, e, at, s["groups"], s["longest"]), s["w"].float().transpose(1, 2))
    return c[e, at].to(s["out"])


def _plain_dgrad(s):
    rows = s["token"].numel()
    e, at = _places(s["offsets"], rows)
    dc = s["dc"].float()
    if rows <= 64:
        return torch.matmul(dc.unsqueeze(1), s["w"][e].float()).squeeze(1).to(s["out"])
    return torch.matmul(_padded(dc, e, at, s["groups"], s["longest"]), s["w"].float())[e, at].to(s["out"])


def _plain_wgrad(s):
    e, at = _places(s["offsets"], s["token"].numel())
    dc = _padded(s["dc"].float(), e, at, s["groups"], s["longest"])
    x = _padded(s["x"][s["token"]].float(), e, at, s["groups"], s["longest"])
    return torch.matmul(dc.transpose(1, 2), x).to(s["out"])


def _plain_combine(s):
    rows = s["o"][s["pos"]].float()
    return (s["shared"].float() + (s["gate"].unsqueeze(2) * rows).sum(1)).to(s["out"])


def _plain_combine_grad(s):
    dy, o = s["dy"].float(), s["o"].float()
    d_o = torch.empty_like(o)
    d_o[s["pos"]] = s["gate"].unsqueeze(2) * dy.unsqueeze(1)
    return d_o.to(s["out"]), (o[s["pos"]] * dy.unsqueeze(1)).sum(2)


def _plain_adapter(s):
    e, at = _places(s["offsets"], s["order"].numel())
    x = _padded(s["x"][s["order"]].float(), e, at, s["groups"], s["longest"])
    h = torch.matmul(x, s["a"].float().transpose(1, 2)) * s["scale"][:, None, None]
    d = torch.matmul(h, s["b"].float().transpose(1, 2))
    y = s["base"].float()
    has = (e < s["groups"]).unsqueeze(1)
    delta = torch.where(has, d[torch.clamp(e, max=s["groups"] - 1), torch.clamp(at, max=s["longest"] - 1)], 0.0)
    return y.index_add(0, s["order"], delta).to(s["out"])


def _plain_adapter_grad(s):
    e, at = _places(s["offsets"], s["order"].numel())
    x = _padded(s["x"][s["order"]].float(), e, at, s["groups"], s["longest"])
    dy = _padded(s["dy"][s["order"]].float(), e, at, s["groups"], s["longest"]) * s["scale"][:, None, None]
    a, b = s["a"].float(), s["b"].float()
    h = torch.matmul(x, a.transpose(1, 2))
    g = torch.matmul(dy, b)
    has = (e < s["groups"]).unsqueeze(1)
    dx = torch.matmul(g, a)[torch.clamp(e, max=s["groups"] - 1), torch.clamp(at, max=s["longest"] - 1)]
    dx = s["dx"].float().index_add(0, s["order"], torch.where(has, dx, 0.0)).to(s["dx"].dtype)
    return dx, torch.matmul(g.transpose(1, 2), x).to(s["out"]), torch.matmul(dy.transpose(1, 2), h).to(s["out"])


_PLAIN = dict(gemm=_plain_gemm, dgrad=_plain_dgrad, wgrad=_plain_wgrad, combine=_plain_combine, combine_grad=_plain_combine_grad,
              adapter=_plain_adapter, adapter_grad=_plain_adapter_grad)


# ------------------------------------------------------------ the package's form
def _own(s):
    import grouped_int4_dequant_amd as moe
    op = s["op"]
    if op == "gemm":
        return moe.grouped_gemm(s["x"], s["w"], s["offsets"], a_row=s["token"], out_dtype=s["out"])
    if op == "dgrad":
        return moe.grouped_gemm_dgrad(s["dc"], s["w"], s["offsets"], out_dtype=s["out"])
    if op == "wgrad":
        return moe.grouped_gemm_wgrad(s["dc"], s["x"], s["offsets"], a_row=s["token"], out_dtype=s["out"])
    if op == "combine":
        return moe.combine(s["o"], s["pos"], weights=s["gate"], add=s["shared"], out_dtype=s["out"])
    if op == "combine_grad":
        return moe.combine_backward(s["dy"], s["o"], s["pos"], s["gate"])
    plan = (s["order"], s["offsets"])
    if op == "adapter":
        return moe.adapter_forward(s["x"], s["a"], s["b"], s["scale"], plan, base=s["base"])
    return moe.adapter_backward(s["dy"], s["x"], s["a"], s["b"], s["scale"], plan, dx_base=s["dx"], grad_dtype=s["out"])


def run(state):
    return _own(state) if own else _PLAIN[state["op"]](state)


def work(case):
    """Each input once, each output once (of the experts or adapters that some row uses)."""
    T, e = case["tokens"], {"bf16": 2, "fp16": 2, "fp32": 4}
    i, o = e[case["type"]], e[case["out"]]
    if case["op"] in ("gemm", "dgrad", "wgrad"):
        G, N, K, P = case["groups"], case["n"], case["k"], T * case["top"]
        used = G * (1.0 - (1.0 - case["top"] / G) ** T)
        moved = {"gemm": T * K * i + used * N * K * i + P * N * o, "dgrad": P * N * i + used * N * K * i + P * K * o,
                 "wgrad": P * N * i + T * K * i + G * N * K * o}[case["op"]]
        return {"bytes": int(moved), "flops": 2 * P * N * K}
    if case["op"] in ("combine", "combine_grad"):
        d, P = case["width"], T * case["top"]
        if case["op"] == "combine":
            return {"bytes": P * d * i + T * d * i + T * d * o + 8 * P, "flops": 2 * P * d}
        return {"bytes": 2 * P * d * i + T * d * i + 12 * P, "flops": 3 * P * d}
    n, N, K, r = case["adapters"], case["n"], case["k"], case["rank"]
    rows = T * (1.0 - case["bare"])
    used = n * (1.0 - (1.0 - 1.0 / n) ** rows)
    if case["op"] == "adapter":
        return {"bytes": int(rows * K * i + used * r * (K + N) * i + 2 * T * N * o), "flops": int(2 * rows * r * (K + N))}
    return {"bytes": int(rows * (K + N) * i + 2 * T * K * i + used * r * (K + N) * i + n * r * (K + N) * o), "flops": int(8 * rows * r * K + 4 * rows * r * (N - K))}


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    op, f8 = s["op"], torch.float64
    if op == "combine":
        y = s["shared"].to(f8)
        for j in range(case["top"]):
            y += s["gate"][:, j, None].to(f8) * s["o"].index_select(0, s["pos"][:, j]).to(f8)
        return y
    if op == "combine_grad":
        d_o = torch.zeros(s["o"].shape, dtype=f8, device="cuda")
        dw = torch.zeros(s["gate"].shape, dtype=f8, device="cuda")
        dy = s["dy"].to(f8)
        for j in range(case["top"]):
            at = s["pos"][:, j].long()
            d_o[at] = s["gate"][:, j, None].to(f8) * dy
            dw[:, j] = (s["o"][at].to(f8) * dy).sum(1)
        return d_o, dw
    ends = s["offsets"].tolist()
    spans = [(e, slice(ends[e], ends[e + 1])) for e in range(s["groups"]) if ends[e + 1] > ends[e]]
    new = lambda *shape: torch.zeros(shape, dtype=f8, device="cuda")  # noqa: E731
    if op == "gemm":
        c = new(case["tokens"] * case["top"], case["n"])
        for e, at in spans:
            c[at] = s["x"][s["token"][at].long()].to(f8) @ s["w"][e].to(f8).t()
        return c
    if op == "dgrad":
        da = new(case["tokens"] * case["top"], case["k"])
        for e, at in spans:
            da[at] = s["dc"][at].to(f8) @ s["w"][e].to(f8)
        return da
    if op == "wgrad":
        dw = new(case["groups"], case["n"], case["k"])
        for e, at in spans:
            dw[e] = s["dc"][at].to(f8).t() @ s["x"][s["token"][at].long()].to(f8)
        return dw
    if op == "adapter":
        y = s["base"].to(f8)
        for e, at in spans:
            rows = s["order"][at].long()
            y[rows] += s["scale"][e].to(f8) * ((s["x"][rows].to(f8) @ s["a"][e].to(f8).t()) @ s["b"][e].to(f8).t())
        return y
    dx, da, db = s["dx"].to(f8), new(*s["a"].shape), new(*s["b"].shape)
    for e, at in spans:
        rows = s["order"][at].long()
        x, dy, a, b = s["x"][rows].to(f8), s["dy"][rows].to(f8) * s["scale"][e].to(f8), s["a"][e].to(f8), s["b"][e].to(f8)
        g = dy @ b
        dx[rows] += g @ a
        da[e] = g.t() @ x
        db[e] = dy.t() @ (x @ a.t())
    return dx, da, db
