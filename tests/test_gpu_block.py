"""The operators of the block around the experts together, as a program runs
them: norm, router, experts and shared expert, gate, residual and the next norm, forward
and backward; in captured graphs, on other streams, with large offsets and used
workspaces."""
import pytest
import torch

import block_reference as R

pytestmark = pytest.mark.gpu

BF, FP, F4 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def moe():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import grouped_int4_dequant_amd as m
    m.load()
    return m


def rnd(g, *shape, dtype=BF, scale=1.0, shift=0.0):
    return (torch.randn(*shape, generator=g) * scale + shift).to(dtype).cuda()


def block(seed, T, d=256, f=64, E=16, k=4, f_sh=96, dtype=BF):
    g = torch.Generator().manual_seed(seed)
    return dict(x=rnd(g, T, d, dtype=F4), w_in=rnd(g, d, dtype=dtype, scale=0.1, shift=1.0), w_r=rnd(g, E, d, scale=d ** -0.5),
                gu=rnd(g, E, 2 * f, d, dtype=dtype, scale=d ** -0.5), dn=rnd(g, E, d, f, dtype=dtype, scale=f ** -0.5), k=k,
                sh_gu=rnd(g, 2 * f_sh, d, dtype=dtype, scale=d ** -0.5), sh_dn=rnd(g, d, f_sh, dtype=dtype, scale=f_sh ** -0.5),
                w_o=rnd(g, d, dtype=dtype, scale=0.1, shift=1.0), gate=rnd(g, d, dtype=dtype, scale=0.3), w_n=rnd(g, d, dtype=dtype, scale=0.1, shift=1.0))


@pytest.mark.parametrize("T", [1, 7, 33])
def test_decode_block(moe, T):
    """Every step against its 64-bit form from what the step before it left."""
    b = block(1, T)
    _, n = moe.residual_norm(None, b["x"], w_n=b["w_in"], dtype=BF)
    value = R.norm(None, b["x"], None, None, 1.0, b["w_in"], 1e-6)[1]
    R.within(n, value[0], R.stored(*value, BF), "norm before")
    logits = moe.router_logits(n, b["w_r"])
    o = moe.few_tokens_layer(n, logits, b["gu"], b["dn"], b["k"], sh_gu=b["sh_gu"], sh_dn=b["sh_dn"])
    v, s, _, _ = R.layer(n, logits, b["gu"], b["dn"], b["k"], b["sh_gu"], b["sh_dn"], None)
    R.within(o, v, R.stored(v, s, BF), "layer")
    y, n2 = moe.residual_norm(o, b["x"], w_o=b["w_o"], gate=b["gate"], w_n=b["w_n"])
    (v, s), after = R.norm(o, b["x"], b["w_o"], b["gate"], 1.0, b["w_n"], 1e-6)
    R.within(y, v, R.stored(v, s, F4), "stream")
    R.within(n2, after[0], R.stored(*after, BF), "norm after")
    # the layer by its parts: grouped products, linear with its activation as the shared expert, combine
    r = moe.route(logits, b["k"])
    shared = moe.linear(moe.linear(n, b["sh_gu"], act="swiglu"), b["sh_dn"])
    gu = moe.grouped_gemm(n, b["gu"], r["offsets"], a_row=r["sorted_token"], out_dtype=F4)
    f = gu.shape[1] // 2
    h = (torch.nn.functional.silu(gu[:, :f]) * gu[:, f:]).to(BF)
    parts = moe.combine(moe.grouped_gemm(h, b["dn"], r["offsets"]), r["pair_pos"].view(T, b["k"]), weights=r["topk_w"], add=shared, out_dtype=F4)
    # the parts round h, each expert's row and the shared row to bf16: 2^-8 of the terms' size each, and the layer's own rounding
    mag = R.layer(n.abs(), logits, b["gu"].abs(), b["dn"].abs(), b["k"], b["sh_gu"].abs(), b["sh_dn"].abs(), None)[0]
    assert ((R.d(parts) - R.d(o)).abs() <= 4 * 2.0 ** -8 * mag).all()


def forward(moe, p, keep):
    _, n = moe.residual_norm(None, p["x"], w_n=p["w_in"], n=keep["n"])
    h = moe.linear(n, p["W1"], bias=p["b1"], act="swiglu", pre=keep["pre"], out=keep["h"])
    o = moe.linear(h, p["W2"], out=keep["o"])
    y, n2 = moe.residual_norm(o, p["x"], w_o=p["w_o"], gate=p["gate"], scale=0.9, w_n=p["w_n"], y=keep["y"], n=keep["n2"])
    return n, h, o, y, n2


def backward(moe, p, keep, dy, dn2, ws):
    dx, d_o, dwo, dg, dwn = moe.residual_norm_backward(dy, dn2, keep["o"], keep["y"], w_o=p["w_o"], gate=p["gate"], scale=0.9, w_n=p["w_n"], grad_dtype=F4, ws=ws[0])
    dh, dW2, _ = moe.linear_backward(d_o, keep["h"], p["W2"], grad_dtype=F4)
    dn, dW1, db1 = moe.linear_backward(dh, keep["n"], p["W1"], pre=keep["pre"], act="swiglu", bias_grad=True, grad_dtype=F4, ws=ws[1])
    din, _, _, _, dwi = moe.residual_norm_backward(dx, dn, None, p["x"], w_n=p["w_in"], grad_dtype=F4, ws=ws[2])
    return dict(x=din, w_in=dwi, W1=dW1, b1=db1, W2=dW2, w_o=dwo, gate=dg, w_n=dwn)


def dense(seed, T, d=128, f=96):
    g = torch.Generator().manual_seed(seed)
    p = dict(x=rnd(g, T, d), w_in=rnd(g, d, scale=0.1, shift=1.0), W1=rnd(g, 2 * f, d, scale=d ** -0.5), b1=rnd(g, 2 * f, scale=0.1),
             W2=rnd(g, d, f, scale=f ** -0.5), w_o=rnd(g, d, scale=0.1, shift=1.0), gate=rnd(g, 4, d, scale=0.5), w_n=rnd(g, d, scale=0.1, shift=1.0))
    new = lambda n: torch.empty(T, n, dtype=BF, device="cuda")  # noqa: E731
    keep = dict(n=new(d), pre=new(2 * f), h=new(f), o=new(d), y=new(d), n2=new(d))
    return p, keep, rnd(g, T, d), rnd(g, T, d)


def workspaces(moe, T, d, f, byte=255):
    sizes = (moe.residual_norm_backward_workspace_bytes(T, d, 4), moe.linear_backward_workspace_bytes(T, 2 * f, d, "swiglu"),
             moe.residual_norm_backward_workspace_bytes(T, d, 1))
    return [torch.full((n,), byte, dtype=torch.uint8, device="cuda") for n in sizes]


def test_dense_block_and_its_gradients(moe):
    """The whole block's gradients against differences of its 64-bit form along random directions."""
    T, d, f = 48, 128, 96
    p, keep, cy, cn = dense(3, T, d, f)
    forward(moe, p, keep)
    grads = backward(moe, p, keep, cy, cn, workspaces(moe, T, d, f))
    base = {n: R.d(t) for n, t in p.items()}

    def loss(v):
        n = R.norm(None, v["x"], None, None, 1.0, v["w_in"], 1e-6)[1][0]
        h = R.linear(n, v["W1"], v["b1"], "swiglu", None)[0]
        (y, _), (m, _) = R.norm(R.linear(h, v["W2"], None, "none", None)[0], v["x"], v["w_o"], v["gate"], 0.9, v["w_n"], 1e-6)
        return (y * R.d(cy)).sum() + (m * R.d(cn)).sum()
    g = torch.Generator().manual_seed(4)
    for name, grad in grads.items():
        way = torch.randn(grad.shape, generator=g, dtype=torch.float64)
        e = 1e-5
        f2 = [float(loss({n: t + s * e * way if n == name else t for n, t in base.items()})) for s in (1, -1)]
        diff, got = (f2[0] - f2[1]) / (2 * e), float((R.d(grad) * way).sum())
        # along the way back some ten tensors are rounded to bf16, 2^-8 of each value at most: each term of the inner
        # product is off by that of its own size and of what was added up in it
        assert abs(diff - got) <= 16 * 2.0 ** -8 * float((R.d(grad).abs() * way.abs()).sum()), (name, diff, got)


def test_workspaces_start_as_anything(moe):
    T, d, f = 72, 128, 96
    p, keep, cy, cn = dense(5, T, d, f)
    forward(moe, p, keep)
    runs = [backward(moe, p, keep, cy, cn, workspaces(moe, T, d, f, byte)) for byte in (0, 255, 127)]
    assert all(torch.equal(runs[0][n], r[n]) for r in runs[1:] for n in r)
    b = block(6, 9)
    n = b["x"].to(BF)
    lg = moe.router_logits(n, b["w_r"])
    size = moe.few_tokens_workspace_bytes(9, BF, 256, 64, 16, 4, 96)
    ys = [moe.few_tokens_layer(n, lg, b["gu"], b["dn"], 4, sh_gu=b["sh_gu"], sh_dn=b["sh_dn"],
                               ws=torch.full((size,), byte, dtype=torch.uint8, device="cuda")) for byte in (0, 255, 127)]
    assert torch.equal(ys[0], ys[1]) and torch.equal(ys[0], ys[2])


@pytest.mark.parametrize("T", [1, 40])
def test_captured_and_replayed(moe, T):
    """A decode block in a graph, replayed on changed inputs with eager work between."""
    b = block(7, T)
    x, n = b["x"], torch.empty(T, 256, dtype=BF, device="cuda")
    lg, o, y, n2 = torch.empty(T, 16, device="cuda"), torch.empty_like(n), torch.empty_like(x), torch.empty_like(n)
    ws = torch.empty(moe.few_tokens_workspace_bytes(T, BF, 256, 64, 16, 4, 96), dtype=torch.uint8, device="cuda")
    h = torch.empty(T, 96, dtype=BF, device="cuda")

    def run(x, n, lg, o, y, n2, h, ws):
        moe.residual_norm(None, x, w_n=b["w_in"], n=n, dtype=BF)
        moe.router_logits(n, b["w_r"], logits=lg)
        moe.few_tokens_layer(n, lg, b["gu"], b["dn"], 4, out=o, ws=ws)
        moe.linear(n, b["sh_gu"], act="swiglu", out=h)
        moe.linear(h, b["sh_dn"], residual=o, out=o)
        moe.residual_norm(o, x, w_o=b["w_o"], gate=b["gate"], w_n=b["w_n"], y=y, n=n2)
    bufs = (x, n, lg, o, y, n2, h, ws)
    run(*bufs)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(*bufs)
    for i in range(4):
        x.copy_(rnd(torch.Generator().manual_seed(20 + i), T, 256, dtype=F4))
        graph.replay()
        got = [t.clone() for t in (o, y, n2)]
        fresh = [x.clone()] + [torch.empty_like(t) for t in bufs[1:]]
        run(*fresh)
        torch.cuda.synchronize()
        assert all(torch.equal(a, e) for a, e in zip(got, (fresh[3], fresh[4], fresh[5]))), i


def test_gradients_captured_and_replayed(moe):
    T, d, f = 96, 128, 96
    p, keep, cy, cn = dense(8, T, d, f)
    ws = workspaces(moe, T, d, f)
    forward(moe, p, keep)
    backward(moe, p, keep, cy, cn, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        forward(moe, p, keep)
        grads = backward(moe, p, keep, cy, cn, ws)
    for i in range(4):
        p["x"].copy_(rnd(torch.Generator().manual_seed(30 + i), T, d))
        cy.copy_(rnd(torch.Generator().manual_seed(40 + i), T, d))
        graph.replay()
        got = {n: t.clone() for n, t in grads.items()}
        _, fresh, _, _ = dense(8, T, d, f)
        forward(moe, p, fresh)
        expect = backward(moe, p, fresh, cy, cn, workspaces(moe, T, d, f))
        torch.cuda.synchronize()
        assert all(torch.equal(got[n], expect[n]) for n in expect), i


def test_on_other_streams(moe):
    T, d, f = 64, 128, 96
    p, keep, cy, cn = dense(9, T, d, f)
    forward(moe, p, keep)
    expect = backward(moe, p, keep, cy, cn, workspaces(moe, T, d, f))
    b = block(10, 5)
    n = b["x"].to(BF)
    lg = moe.router_logits(n, b["w_r"])
    o = moe.few_tokens_layer(n, lg, b["gu"], b["dn"], 4)
    torch.cuda.synchronize()
    sides = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s in sides:  # both at once, each with workspaces of its own
        with torch.cuda.stream(s):
            got.append(backward(moe, p, keep, cy, cn, workspaces(moe, T, d, f)))
    given = moe.few_tokens_layer(n, lg, b["gu"], b["dn"], 4, stream=sides[0])
    lin = moe.linear(keep["n"], p["W1"], bias=p["b1"], act="swiglu", stream=sides[1])
    y, _ = moe.residual_norm(keep["o"], p["x"], w_o=p["w_o"], gate=p["gate"], scale=0.9, stream=sides[0])
    torch.cuda.synchronize()
    assert all(torch.equal(g[k], expect[k]) for g in got for k in expect)
    assert torch.equal(given, o) and torch.equal(lin, keep["h"]) and torch.equal(y, keep["y"])


def test_offsets_beyond_32_bits(moe):
    """Rows and experts whose elements lie past 2^32 bytes and 2^31 elements."""
    T, d = 1100000, 2048
    x = torch.zeros(T, d, dtype=BF, device="cuda")
    g = torch.Generator().manual_seed(11)
    tail = rnd(g, 300, d)
    x[-300:] = tail
    w, W = rnd(g, d, shift=1.0), rnd(g, 64, d, scale=d ** -0.5)
    y, n = moe.residual_norm(x, x, w_o=w, w_n=w)
    ey, en = moe.residual_norm(tail, tail, w_o=w, w_n=w)
    assert torch.equal(y[-300:], ey) and torch.equal(n[-300:], en) and (y[:5] == 0).all()
    del y, n
    z = moe.linear(x, W)
    assert torch.equal(z[-256:], moe.linear(x[-16640:].clone(), W)[-256:])
    dz = torch.zeros_like(z)
    dz[-300:] = rnd(g, 300, 64)
    dx, dW, _ = moe.linear_backward(dz, x, W, grad_dtype=F4)
    value = R.linear_grad(dz[-300:], tail, W, None, "none", BF)
    R.within(dW, value[1][0], R.stored(*value[1], F4), "dW")
    R.within(dx[-300:], value[0][0], R.stored(*value[0], BF), "dx")
    del dx, z
    gx, go, dwo, _, dwn = moe.residual_norm_backward(x, x, x, x, w_o=w, w_n=w, grad_dtype=F4)
    e = moe.residual_norm_backward(tail, tail, tail, tail, w_o=w, w_n=w, grad_dtype=F4)
    assert torch.equal(gx[-300:], e[0]) and torch.equal(go[-300:], e[1])
    value = R.norm_grad(tail, tail, tail, tail, w, None, 1.0, w, 1e-6)
    R.within(dwo, value["dw_o"][0], R.stored(value["dw_o"][0], value["dw_o"][1] + R.sums(T, 0 * value["dw_o"][0]), F4), "dw_o")
    del gx, go, x
    torch.cuda.empty_cache()
    E, d, f = 200, 4096, 2048
    gu, dn = torch.zeros(E, 2 * f, d, dtype=BF, device="cuda"), torch.zeros(E, d, f, dtype=BF, device="cuda")
    last_gu, last_dn = rnd(g, 1, 2 * f, d, scale=d ** -0.5), rnd(g, 1, d, f, scale=f ** -0.5)
    gu[-1:], dn[-1:] = last_gu, last_dn
    xs, lg = rnd(g, 3, d), torch.zeros(3, E, device="cuda")
    lg[:, -1] = 1.0
    got = moe.few_tokens_layer(xs, lg, gu, dn, 1)
    assert torch.equal(got, moe.few_tokens_layer(xs, lg[:, -1:].contiguous(), last_gu, last_dn, 1)) and got.abs().max() > 0
