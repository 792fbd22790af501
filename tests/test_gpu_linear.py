"""The product with bias, activation and residual and its gradients on the GPU
against plain 64-bit forms, element by element."""
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


def rnd(g, *shape, dtype=BF, scale=1.0):
    return (torch.randn(*shape, generator=g) * scale).to(dtype).cuda()


def wider(t, extra, fill):
    """The same values as a view of a matrix with `extra` more columns, which hold `fill`."""
    w = torch.full((t.shape[0], t.shape[1] + extra), fill, dtype=t.dtype, device=t.device)
    w[:, :t.shape[1]] = t
    return w, w[:, :t.shape[1]]


ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh", "swiglu", "geglu")
#         T, N, K: each kernel form, whole and ragged tiles, sizes of no alignment
SHAPES = {"one": (1, 1, 1), "two": (1, 2, 8), "decode": (1, 264, 520), "few16": (16, 72, 136), "few17": (17, 40, 1544), "few33": (33, 264, 200),
          "few64": (64, 136, 64), "small65": (65, 128, 72), "small": (129, 200, 328), "odd": (77, 66, 131), "odd_one": (1, 34, 77),
          "odd_k": (70, 64, 67), "wide128": (200, 33032, 72), "wide256": (1290, 6672, 200),
          "wide_dx": (1290, 264, 6672), "wide_dW": (200, 2824, 2824),
          "long": (8200, 136, 72), "long_odd": (5003, 70, 33), "long_wide": (4100, 520, 776)}  # rows cut into parts for dW


def problem(shape, act, dtype, out, bias=None, residual=False, pre=False, seed=1):
    T, N, K = SHAPES[shape]
    g = torch.Generator().manual_seed(seed)
    N = N + N % 2 if act in R.GATED else N
    cols = N // 2 if act in R.GATED else N
    p = dict(x=rnd(g, T, K, dtype=dtype), W=rnd(g, N, K, dtype=dtype, scale=K ** -0.5))
    p["bias"] = None if bias is None else rnd(g, N, dtype=bias)
    p["residual"] = rnd(g, T, cols, dtype=out) if residual else None
    p["pre"] = torch.full((T, N), 5.0, dtype=dtype, device="cuda") if pre else None
    return p, T, N, K, cols


CASES = [("small", a, BF, BF, BF, True, True) for a in ACTS] + [("few17", a, FP, F4, F4, False, True) for a in ACTS]
CASES += [("odd", a, FP, FP, FP, True, True) for a in ACTS] + [("wide256", a, BF, BF, None, False, True) for a in ("none", "gelu", "swiglu")]
CASES += [(s, a, BF, F4, BF, True, False) for s in SHAPES for a in ("silu", "swiglu")]
CASES += [("wide256", "geglu", FP, F4, FP, True, True), ("wide128", "gelu", FP, FP, F4, True, True), ("wide128", "none", BF, F4, None, False, False)]


@pytest.mark.parametrize("shape,act,dtype,out,bias,residual,pre", CASES,
                         ids=["-".join([c[0], c[1], str(c[2])[6:], str(c[3])[6:], str(i)]) for i, c in enumerate(CASES)])
def test_forward(moe, shape, act, dtype, out, bias, residual, pre):
    p, T, N, K, cols = problem(shape, act, dtype, out, bias, residual, pre)
    y = moe.linear(p["x"], p["W"], bias=p["bias"], act=act, residual=p["residual"], out_dtype=out, pre=p["pre"])
    value, slack, z, zs = R.linear(p["x"], p["W"], p["bias"], act, p["residual"])
    R.within(y, value, R.stored(value, slack, out), "y")
    if pre:
        R.within(p["pre"], z, R.stored(z, zs, dtype), "pre")
    assert torch.equal(y, moe.linear(p["x"], p["W"], bias=p["bias"], act=act, residual=p["residual"], out_dtype=out))


@pytest.mark.parametrize("shape,act", [("few33", "swiglu"), ("small", "gelu"), ("odd", "geglu"), ("wide128", "silu"), ("wide256", "swiglu"), ("decode", "none")])
def test_strided_and_in_place(moe, shape, act):
    p, T, N, K, cols = problem(shape, act, BF, BF, BF, True, True)
    expect = moe.linear(p["x"], p["W"], bias=p["bias"], act=act, residual=p["residual"], pre=p["pre"])
    (xw, x), (rw, r), (pw, pre) = wider(p["x"], 8, float("nan")), wider(p["residual"], 5, 3.0), wider(torch.zeros_like(p["pre"]), 3, 2.0)
    got = moe.linear(x, p["W"], bias=p["bias"], act=act, residual=r, out=r, pre=pre)
    assert got.data_ptr() == r.data_ptr() and torch.equal(got, expect) and torch.equal(pre, p["pre"])
    assert (rw[:, cols:] == 3).all() and (pw[:, N:] == 2).all()
    # an odd row stride: rows of no 16-byte alignment
    (_, x), (rw, r) = wider(p["x"], 1, float("nan")), wider(torch.zeros_like(expect), 1, 4.0)
    got = moe.linear(x, p["W"], bias=p["bias"], act=act, residual=p["residual"], out=r)
    value, slack, _, _ = R.linear(p["x"], p["W"], p["bias"], act, p["residual"])
    R.within(got, value, R.stored(value, slack, BF), "odd stride")
    assert (rw[:, cols:] == 4).all()


GRADS = [("small", a, BF, BF, True) for a in ACTS] + [("odd", a, FP, F4, True) for a in ACTS] + [("few33", a, FP, FP, True) for a in ("none", "gelu", "swiglu")]
GRADS += [(s, a, BF, F4, True) for s in SHAPES for a in ("none", "swiglu")] + [("wide256", "geglu", FP, FP, False), ("wide128", "gelu_tanh", BF, BF, True)]


@pytest.mark.parametrize("shape,act,dtype,grad,bias", GRADS, ids=["-".join([c[0], c[1], str(c[2])[6:], str(c[3])[6:], str(i)]) for i, c in enumerate(GRADS)])
def test_gradients(moe, shape, act, dtype, grad, bias):
    p, T, N, K, cols = problem(shape, act, dtype, dtype, seed=3)
    g = torch.Generator().manual_seed(4)
    dy, pre = rnd(g, T, cols, dtype=dtype), rnd(g, T, N, dtype=dtype) if act != "none" else None
    got = moe.linear_backward(dy, p["x"], p["W"], pre=pre, act=act, bias_grad=bias, grad_dtype=grad)
    parts = R.linear_grad(dy, p["x"], p["W"], pre, act, dtype)
    for v, (value, slack), name, t in zip(got, parts, ("dx", "dW", "db"), (dtype, grad, grad)):
        if v is not None:
            R.within(v, value, R.stored(value, slack, t), name)
    assert (got[2] is not None) == bias
    again = moe.linear_backward(dy, p["x"], p["W"], pre=pre, act=act, bias_grad=bias, grad_dtype=grad)
    assert all(a is b or torch.equal(a, b) for a, b in zip(got, again))


@pytest.mark.parametrize("shape,act", [("small", "swiglu"), ("odd", "gelu"), ("few17", "none"), ("wide256", "silu")])
def test_gradients_accumulate_and_strides(moe, shape, act):
    p, T, N, K, cols = problem(shape, act, BF, BF, seed=5)
    g = torch.Generator().manual_seed(6)
    dy, pre = rnd(g, T, cols), rnd(g, T, N)
    fresh = moe.linear_backward(dy, p["x"], p["W"], pre=pre, act=act, bias_grad=True, grad_dtype=F4)
    dW, db = rnd(g, N, K, dtype=F4), rnd(g, N, dtype=F4)
    sum_w, sum_b = dW + fresh[1], db + fresh[2]
    (_, dyv), (_, xv), (_, prev) = wider(dy, 8, float("nan")), wider(p["x"], 8, float("nan")), wider(pre, 8, float("nan"))
    dxw, dx = wider(torch.zeros(T, K, dtype=F4, device="cuda"), 3, 9.0)
    got = moe.linear_backward(dyv, xv, p["W"], pre=prev, act=act, dx=dx, dW=dW, db=db, accumulate=True)
    assert torch.equal(got[1], sum_w) and torch.equal(got[2], sum_b) and got[1] is dW and got[2] is db
    (value, slack), _, _ = R.linear_grad(dy, p["x"], p["W"], pre, act, BF)
    R.within(dx, value, R.stored(value, slack, F4), "dx fp32")
    assert (dxw[:, K:] == 9).all()


def test_gradients_against_differences(moe):
    """d loss / d parameter along a direction, loss = <y, c>, by central differences of the 64-bit form and by the call."""
    T, N, K = 24, 48, 40
    g = torch.Generator().manual_seed(7)
    x, W, b, c = rnd(g, T, K), rnd(g, N, K, scale=K ** -0.5), rnd(g, N), rnd(g, T, N // 2)
    pre = torch.empty(T, N, dtype=BF, device="cuda")
    moe.linear(x, W, bias=b, act="swiglu", pre=pre)
    dx, dW, db = moe.linear_backward(c, x, W, pre=pre, act="swiglu", bias_grad=True, grad_dtype=F4)
    X, V, Bv, Cv = (R.d(t) for t in (x, W, b, c))
    for which, grad in ((0, dx), (1, dW), (2, db)):
        way = torch.randn(grad.shape, generator=g, dtype=torch.float64)
        h = 1e-5
        f = [(R.linear(*[t + s * h * way if i == which else t for i, t in enumerate((X, V, Bv))], "swiglu", None)[0] * Cv).sum() for s in (1, -1)]
        diff = float((f[0] - f[1]) / (2 * h))
        # pre is rounded to bf16 (2^-8 of each of its values, which are about 1.4) and dz again: every term of the
        # inner product with the direction is off by a few 2^-8 of its size
        mag = float((R.d(grad).abs() * way.abs()).sum())
        assert abs(diff - float((R.d(grad) * way).sum())) <= 4 * 2.0 ** -8 * mag, which


def test_no_rows(moe):
    x, W = torch.empty(0, 16, dtype=BF, device="cuda"), torch.ones(8, 16, dtype=BF, device="cuda")
    assert moe.linear(x, W, act="swiglu").shape == (0, 4)
    dW, db = torch.full((8, 16), 3.0, device="cuda"), torch.full((8,), 3.0, device="cuda")
    dx, a, b = moe.linear_backward(torch.empty(0, 8, dtype=BF, device="cuda"), x, W, bias_grad=True, grad_dtype=F4)
    assert dx.shape == (0, 16) and (a == 0).all() and (b == 0).all()
    moe.linear_backward(torch.empty(0, 8, dtype=BF, device="cuda"), x, W, dW=dW, db=db, accumulate=True)
    assert (dW == 3).all() and (db == 3).all()


@pytest.mark.parametrize("shape", ["few16", "small", "odd", "wide128"])
def test_infinities_and_nan_stay_in_their_rows(moe, shape):
    p, T, N, K, cols = problem(shape, "silu", BF, F4)
    clean = moe.linear(p["x"], p["W"], act="silu", out_dtype=F4)
    x = p["x"].clone()
    x[T // 2, K // 2] = float("nan")
    x[0, 0] = float("inf")
    got = moe.linear(x, p["W"], act="silu", out_dtype=F4)
    assert torch.isnan(got[T // 2]).all() and not torch.isfinite(got[0]).any() | (got[0] == 0).any()
    rest = [t for t in range(T) if t not in (0, T // 2)]
    assert torch.equal(got[rest], clean[rest])


@pytest.mark.parametrize("act", ACTS[1:5])
def test_activations_far_from_zero(moe, act):
    """z = x (W = 1) over all of bf16's magnitudes, forward and gradient; finite wherever the formula is."""
    z = torch.cat([s * torch.logspace(-38, 38, 153, dtype=torch.float64) for s in (1, -1)]).to(BF).cuda()[:, None]
    one = torch.ones(1, 1, dtype=BF, device="cuda")
    got = moe.linear(z, one, act=act, out_dtype=F4)
    value = R.curve(act, R.d(z))
    R.within(got, value, R.stored(value, R.curve_slack(act, R.d(z).clamp(-30, 30), value) + 2 * R.U * value.abs(), F4), act)
    dy = torch.ones_like(z)
    dx, dW, db = moe.linear_backward(dy, torch.ones_like(z), one, pre=z, act=act)
    value = torch.nan_to_num(R.slope(act, R.d(z)))
    R.within(dx, value, R.stored(value, R.slope_slack(act, R.d(z).clamp(-30, 30)), BF) * (1 + 2.0 ** -7), act)
