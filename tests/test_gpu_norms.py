"""The norms before and after a block with gate and residual, and their
gradients, on the GPU against plain 64-bit forms, element by element."""
import pytest
import torch

import block_reference as R

pytestmark = pytest.mark.gpu

BF, FP, F4 = torch.bfloat16, torch.float16, torch.float32
EPS = 1e-6


@pytest.fixture(scope="module")
def moe():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import grouped_int4_dequant_amd as m
    m.load()
    return m


def rnd(g, *shape, dtype=BF, scale=1.0, shift=0.0):
    return (torch.randn(*shape, generator=g) * scale + shift).to(dtype).cuda()


#        rows, width, rows of gate (0: none)
SHAPES = {"one": (1, 1, 1), "row": (1, 2048, 0), "tiny": (3, 7, 3), "w512": (37, 512, 1), "w513": (30, 513, 5), "w1024": (9, 1000, 9), "w2048": (1030, 2048, 1),
          "w2049": (12, 2049, 2), "w4096": (6, 4096, 3), "w8192": (5, 8192, 1), "w8193": (4, 8193, 4), "max": (3, 16384, 1),
          "sequences": (1300, 264, 13), "tokens": (700, 72, 700), "pairs": (1400, 40, 700), "short": (2600, 33, 520)}


def problem(shape, dtype, stream, weights, seed=1):
    T, d, gates = SHAPES[shape]
    g = torch.Generator().manual_seed(seed)
    return dict(o=rnd(g, T, d, dtype=dtype, scale=2.0), x=rnd(g, T, d, dtype=stream), w_o=rnd(g, d, dtype=weights, scale=0.2, shift=1.0),
                gate=rnd(g, gates, d, dtype=weights, scale=0.5) if gates else None, w_n=rnd(g, d, dtype=weights, scale=0.2, shift=1.0),
                dy=rnd(g, T, d, dtype=stream), dn=rnd(g, T, d, dtype=dtype), y=rnd(g, T, d, dtype=stream, scale=1.5))


TYPES = [(BF, BF, BF), (FP, F4, F4), (BF, F4, BF), (FP, FP, F4)]
CASES = [(s, *TYPES[i % 4]) for i, s in enumerate(SHAPES)] + [("w2048", *t) for t in TYPES] + [("sequences", *t) for t in TYPES]
PARTS = [("all", {}), ("add", dict(w_o=None, gate=None)), ("gate", dict(w_o=None, w_n=None)), ("post", dict(gate=None, w_n=None)), ("before", dict(o=None)),
         ("alone", dict(x=None))]


def ids(cases):
    return ["-".join([c[0], *[str(t)[6:] for t in c[1:4]], str(i)]) for i, c in enumerate(cases)]


@pytest.mark.parametrize("parts", [p for _, p in PARTS], ids=[n for n, _ in PARTS])
@pytest.mark.parametrize("shape,dtype,stream,weights", CASES, ids=ids(CASES))
def test_forward(moe, shape, dtype, stream, weights, parts):
    p = dict(problem(shape, dtype, stream, weights), **parts)
    scale = 0.75 if p["o"] is not None else 1.0
    gate = None if p["o"] is None else p["gate"]
    y, n = moe.residual_norm(p["o"], p["x"], w_o=p["w_o"], gate=gate, scale=scale, w_n=p["w_n"], eps=EPS,
                             dtype=dtype if p["o"] is None else None)
    (v, vs), after = R.norm(p["o"], p["x"], p["w_o"], gate, scale, p["w_n"], EPS)
    if p["o"] is None:
        assert y is None
    else:
        assert y.dtype == (dtype if p["x"] is None else stream)
        R.within(y, v, R.stored(v, vs, y.dtype), "y")
    if p["w_n"] is None:
        assert n is None
    else:
        assert n.dtype == dtype
        R.within(n, after[0], R.stored(*after, dtype), "n")


@pytest.mark.parametrize("parts", [p for n, p in PARTS if n != "alone"], ids=[n for n, _ in PARTS if n != "alone"])
@pytest.mark.parametrize("shape,dtype,stream,weights", CASES, ids=ids(CASES))
def test_gradients(moe, shape, dtype, stream, weights, parts):
    p = dict(problem(shape, dtype, stream, weights), **parts)
    dn = None if p["w_n"] is None else p["dn"]
    args = (p["dy"], dn, p["o"], p["y"])
    more = dict(w_o=p["w_o"], gate=p["gate"], scale=0.75, w_n=p["w_n"], eps=EPS)
    got = dict(zip(("dx", "d_o", "dw_o", "dgate", "dw_n"), moe.residual_norm_backward(*args, **more, grad_dtype=F4)))
    if p["o"] is None:
        more.update(w_o=None, gate=None)
    expect = R.norm_grad(*args, *more.values())
    assert {k for k, v in got.items() if v is not None} == set(expect)
    types = dict(dx=stream, d_o=dtype)
    for name, (value, slack) in expect.items():
        t = types.get(name, F4)
        assert got[name].dtype == t
        R.within(got[name], value, R.stored(value, slack, t), name)
    again = moe.residual_norm_backward(*args, **dict(more, w_o=p["w_o"], gate=p["gate"]), grad_dtype=F4)
    assert all(b is None or torch.equal(got[k], b) for k, b in zip(("dx", "d_o", "dw_o", "dgate", "dw_n"), again))


@pytest.mark.parametrize("shape", ["w513", "w2048", "sequences", "tokens", "short"])
def test_gradients_rounded_and_accumulated(moe, shape):
    p = problem(shape, BF, BF, BF, seed=2)
    args, more = (p["dy"], p["dn"], p["o"], p["y"]), dict(w_o=p["w_o"], gate=p["gate"], scale=1.0, w_n=p["w_n"], eps=EPS)
    fresh = moe.residual_norm_backward(*args, **more, grad_dtype=F4)
    low = moe.residual_norm_backward(*args, **more)
    for a, b in zip(fresh[2:], low[2:]):
        assert b.dtype == BF and torch.equal(a.to(BF), b)
    held = [torch.randn_like(t) for t in fresh[2:]]
    sums = [a + b for a, b in zip(held, fresh[2:])]
    moe.residual_norm_backward(*args, **more, dw_o=held[0], dgate=held[1], dw_n=held[2], grad_dtype=F4, accumulate=True)
    assert all(torch.equal(a, b) for a, b in zip(held, sums))


def test_strided_and_in_place(moe):
    for shape in ("w513", "w2048", "w8192"):
        p = problem(shape, BF, F4, BF, seed=3)
        T, d = p["o"].shape
        y, n = moe.residual_norm(p["o"], p["x"], w_o=p["w_o"], gate=p["gate"], w_n=p["w_n"])

        def wider(t, extra):
            w = torch.full((T, d + extra), 7.0, dtype=t.dtype, device="cuda")
            w[:, :d] = t
            return w, w[:, :d]
        (ow, o), (xw, x) = wider(p["o"], 3), wider(p["x"], 1)
        got = moe.residual_norm(o, x, w_o=p["w_o"], gate=p["gate"], w_n=p["w_n"], y=x, n=o)
        assert torch.equal(x, y) and torch.equal(o, n) and got[0] is x and got[1] is o
        assert (ow[:, d:] == 7).all() and (xw[:, d:] == 7).all()
        more = dict(w_o=p["w_o"], gate=p["gate"], w_n=p["w_n"])
        expect = moe.residual_norm_backward(p["dy"], p["dn"], p["o"], p["y"], **more)
        (gw, dy), (_, dn), (_, ov), (_, yv) = wider(p["dy"], 5), wider(p["dn"], 1), wider(p["o"], 2), wider(p["y"], 3)
        dw, d_o = wider(torch.zeros_like(p["o"]), 1)
        got = moe.residual_norm_backward(dy, dn, ov, yv, **more, dx=dy, d_o=d_o)
        assert all(torch.equal(a, b) for a, b in zip(got, expect))
        assert (gw[:, d:] == 7).all() and (dw[:, d:] == 7).all()


def test_only_dn(moe):
    p = problem("w513", BF, BF, BF, seed=4)
    got = moe.residual_norm_backward(None, p["dn"], None, p["y"], w_n=p["w_n"])
    expect = moe.residual_norm_backward(torch.zeros_like(p["y"]), p["dn"], None, p["y"], w_n=p["w_n"])
    assert all(a is b or torch.equal(a, b) for a, b in zip(got, expect))


def test_no_rows(moe):
    e = torch.empty(0, 64, dtype=BF, device="cuda")
    w = torch.ones(64, dtype=BF, device="cuda")
    y, n = moe.residual_norm(e, e, w_o=w, gate=torch.ones(3, 64, dtype=BF, device="cuda"), w_n=w)
    assert y.shape == n.shape == (0, 64)
    out = moe.residual_norm_backward(e, e, e, e, w_o=w, gate=torch.ones(3, 64, dtype=BF, device="cuda"), w_n=w, grad_dtype=F4)
    assert all((g == 0).all() for g in out[2:]) and out[3].shape == (3, 64)
    held = [torch.full(s, 3.0, device="cuda") for s in ((64,), (3, 64), (64,))]
    moe.residual_norm_backward(e, e, e, e, w_o=w, gate=torch.ones(3, 64, dtype=BF, device="cuda"), w_n=w, dw_o=held[0], dgate=held[1], dw_n=held[2],
                               grad_dtype=F4, accumulate=True)
    assert all((g == 3).all() for g in held)


@pytest.mark.parametrize("shape", ["w513", "w2048", "w8192"])
def test_rows_are_apart(moe, shape):
    """Infinities, NaN and zeros in one row touch that row alone (and, in the gradient, the column sums)."""
    p = problem(shape, BF, BF, BF, seed=5)
    more = dict(w_o=p["w_o"], gate=p["gate"], w_n=p["w_n"])
    clean = moe.residual_norm(p["o"], p["x"], **more)
    o, x = p["o"].clone(), p["x"].clone()
    o[1, 3], o[2] = float("nan"), 0.0
    x[1, 5], x[2] = float("inf"), 0.0
    got = moe.residual_norm(o, x, **more)
    rest = [t for t in range(o.shape[0]) if t not in (1, 2)]
    for a, b in zip(got, clean):
        assert torch.equal(a[rest], b[rest]) and torch.isnan(a[1]).any() and (a[2] == 0).all()
    dx, d_o = moe.residual_norm_backward(p["dy"], p["dn"], p["o"], p["y"], **more)[:2]
    y, dy = p["y"].clone(), p["dy"].clone()
    y[1, 0], dy[1, 2] = float("nan"), float("inf")
    gx, go = moe.residual_norm_backward(dy, p["dn"], p["o"], y, **more)[:2]
    rest = [t for t in range(o.shape[0]) if t != 1]
    assert torch.equal(gx[rest], dx[rest]) and torch.equal(go[rest], d_o[rest]) and torch.isnan(gx[1]).any()


def test_gradients_against_differences(moe):
    T, d = 24, 40
    g = torch.Generator().manual_seed(7)
    o, x, wo, gate, wn = rnd(g, T, d), rnd(g, T, d, dtype=F4), rnd(g, d, dtype=F4, shift=1.0), rnd(g, 3, d, dtype=F4), rnd(g, d, dtype=F4, shift=1.0)
    cy, cn = rnd(g, T, d, dtype=F4), rnd(g, T, d)
    y, _ = moe.residual_norm(o, x, w_o=wo, gate=gate, scale=0.5, w_n=wn)
    dx, d_o, dwo, dgate, dwn = moe.residual_norm_backward(cy, cn, o, y, w_o=wo, gate=gate, scale=0.5, w_n=wn)
    base = [R.d(t) for t in (o, x, wo, gate, wn)]

    def loss(vals):
        (v, _), (n, _) = R.norm(vals[0], vals[1], vals[2], vals[3], 0.5, vals[4], EPS)
        return (v * R.d(cy)).sum() + (n * R.d(cn)).sum()
    for which, grad in enumerate((d_o, dx, dwo, dgate, dwn)):
        way = torch.randn(grad.shape, generator=g, dtype=torch.float64)
        h = 1e-5
        f = [loss([t + s * h * way if i == which else t for i, t in enumerate(base)]) for s in (1, -1)]
        diff, mag = float((f[0] - f[1]) / (2 * h)), float((R.d(grad).abs() * way.abs()).sum())
        # d_o is stored in bf16 (half a step of each value); the others are fp32 sums; the differences' own error is about h^2
        assert abs(diff - float((R.d(grad) * way).sum())) <= (2.0 ** -8 if which == 0 else 2.0 ** -16) * mag, which
