"""Gradients of a product with an activation: what of dz, the gradient at the product, enters dx = dz W and dW = dz^T x.
Against 64 bits, element by element.

dz is formed in fp32 (block_reference.act_grad gives its slack) and enters as a sum of 16-bit parts of its own sign. Three bf16
parts hold 24 bits: all of it, for fp32 results. Of two parts the first holds a value cut to the type's bits (or the next smaller
one), the second what is left: bf16 8 + 8 bits, cut where a third part follows, so 2^-15 of dz at most is lost; fp16
11 + 11 bits, the second rounded, so 2^-22, or half of fp16's smallest step, 2^-25, in each element. (fp16 with an fp32 result
beside it takes bf16 parts.) An fp16 operand is exactly two bf16 parts. Every pair of parts adds a term to the sum.
"""
import pytest
import torch

import block_reference as R

pytestmark = pytest.mark.gpu

BF, FP, F4 = torch.bfloat16, torch.float16, torch.float32
ACTS = ("relu", "silu", "gelu", "gelu_tanh", "swiglu", "geglu")
#         T, N, K: few rows, small tiles, rows of no alignment, rows of dW cut into parts, tiles of 128 and 256 rows
SHAPES = {"one": (1, 2, 1), "few": (33, 264, 200), "few_long": (20, 1544, 136), "small": (129, 200, 328), "odd": (77, 66, 131), "odd_few": (9, 70, 33),
          "wide_dx128": (700, 264, 6672), "wide_dx256": (1290, 328, 6672), "wide_dW": (200, 2824, 2824), "cut": (8200, 136, 72), "cut_odd": (5003, 70, 33),
          "cut_wide": (4100, 520, 776)}
RESULTS = {"16": (None, None), "dW32": (None, F4), "dx32": (F4, None), "32": (F4, F4)}


@pytest.fixture(scope="module")
def moe():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import grouped_int4_dequant_amd as m
    m.load()
    return m


def rnd(g, *shape, dtype=BF, scale=1.0):
    return (torch.randn(*shape, generator=g) * scale).to(dtype).cuda()


def problem(shape, act, dtype, seed=1):
    T, N, K = SHAPES[shape]
    g = torch.Generator().manual_seed(seed)
    cols = N // 2 if act in R.GATED else N
    return rnd(g, T, cols, dtype=dtype), rnd(g, T, K, dtype=dtype), rnd(g, N, K, dtype=dtype, scale=K ** -0.5), rnd(g, T, N, dtype=dtype)


def given(x, dx):
    return None if dx is None else torch.empty(x.shape, dtype=dx, device="cuda")


def reference(dy, x, W, pre, act, dtype, dx, dW):
    dz, s32, _ = R.act_grad(dy, pre, act, dtype)
    x, W = R.d(x), R.d(W)
    any32 = dx is F4 or dW is F4

    def slack(result, terms):
        if result is F4:
            return s32, 6 * terms
        cut = 2.0 ** -22 * dz.abs() + 2.0 ** -25 if dtype is FP and not any32 else 2.0 ** -15 * dz.abs()
        return s32 + cut, 4 * terms
    (sx, nx), (sw, nw) = slack(dx, dz.shape[1]), slack(dW, dz.shape[0])
    return ((dz @ W, sx @ W.abs() + R.sums(nx, dz.abs() @ W.abs())), (dz.T @ x, sw.T @ x.abs() + R.sums(nw, dz.abs().T @ x.abs())),
            (dz.sum(0), s32.sum(0) + R.sums(dz.shape[0], dz.abs().sum(0))))


CASES = [("small", a, t, r) for a in ACTS for t in (BF, FP) for r in RESULTS] + [(s, a, t, r) for s in SHAPES if s != "small" for a, t, r in (
    ("swiglu", BF, "16"), ("silu", BF, "dW32"), ("geglu", FP, "16"), ("relu", FP, "32"), ("gelu", BF, "32"), ("swiglu", FP, "dx32"))]


@pytest.mark.parametrize("shape,act,dtype,results", CASES, ids=[f"{s}-{a}-{str(t)[6:]}-{r}" for s, a, t, r in CASES])
def test_rounded_once(moe, shape, act, dtype, results):
    dy, x, W, pre = problem(shape, act, dtype)
    tx, tw = RESULTS[results]
    got = moe.linear_backward(dy, x, W, pre=pre, act=act, bias_grad=True, dx=given(x, tx), grad_dtype=tw)
    for v, (value, slack), t, name in zip(got, reference(dy, x, W, pre, act, dtype, tx, tw), (tx, tw, tw), ("dx", "dW", "db")):
        assert v.dtype is (t or dtype)
        R.within(v, value, R.stored(value, slack, v.dtype), name)
    again = moe.linear_backward(dy, x, W, pre=pre, act=act, bias_grad=True, dx=given(x, tx), grad_dtype=tw)
    assert all(torch.equal(a, b) for a, b in zip(got, again))


@pytest.mark.parametrize("shape", ["few", "small", "odd", "wide_dx128", "cut"])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_dz_of_any_size(moe, shape, dtype):
    """fp32 results of terms from 2^-30 to 2^30, both within fp16's range as dy and pre: columns of dz far apart, each column's weights as far."""
    dy, x, W, pre = problem(shape, "swiglu", dtype, seed=2)
    T, N, K = SHAPES[shape]
    h = N // 2
    step = (2.0 ** (15.0 * ((torch.arange(h) % 3) - 1))).to(dtype).cuda()
    dy, pre = (dy * step).clamp(-60000, 60000), torch.cat([pre[:, :h], (pre[:, h:] * step).clamp(-60000, 60000)], 1)
    got = moe.linear_backward(dy, x, W, pre=pre, act="swiglu", dx=given(x, F4), grad_dtype=F4, bias_grad=True)
    for v, (value, slack), name in zip(got, reference(dy, x, W, pre, "swiglu", dtype, F4, F4), ("dx", "dW", "db")):
        R.within(v, value, R.stored(value, slack, F4), name)


@pytest.mark.parametrize("results", RESULTS)
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("shape", ["few", "small", "odd", "wide_dx128", "wide_dW"])
def test_infinities(moe, shape, dtype, results):
    """Infinite weights, inputs and dy give the formula's infinities and NaN, and only there (relu: dz is dy, so that its first part would hold it whole, or zero)."""
    dy, x, W, pre = problem(shape, "relu", dtype, seed=3)
    T, N, K = SHAPES[shape]
    tx, tw = RESULTS[results]

    def call(dy, x, W):
        return moe.linear_backward(dy, x, W, pre=pre, act="relu", dx=given(x, tx), grad_dtype=tw)[:2]
    clean = call(dy, x, W)
    dz = torch.where(pre > 0, dy, 0.0)
    w = W.clone()
    w[N // 3, 5], w[N - 1, 7], w[2, 9] = float("inf"), -float("inf"), float("nan")
    dx, dW = call(dy, x, w)
    rest = [k for k in range(K) if k not in (5, 7, 9)]
    assert torch.equal(dx[:, rest], clean[0][:, rest]) and torch.equal(dW, clean[1]) and torch.isnan(dx[:, 9]).all()
    for n, k, sign in ((N // 3, 5, 1), (N - 1, 7, -1)):
        expect = R.d(dz[:, n]) * sign * float("inf")  # NaN where dz is zero
        assert torch.equal(R.d(dx[:, k]).nan_to_num(0.0, 1.0, -1.0), expect.nan_to_num(0.0, 1.0, -1.0))
        assert torch.equal(torch.isnan(dx[:, k]).cpu(), torch.isnan(expect))
    v = x.clone()
    v[T // 2, 3] = -float("inf")
    dx, dW = call(dy, v, W)
    expect = R.d(dz[T // 2]) * -float("inf")
    rest = [k for k in range(K) if k != 3]
    assert torch.equal(dx, clean[0]) and torch.equal(dW[:, rest], clean[1][:, rest])
    assert torch.equal(R.d(dW[:, 3]).nan_to_num(0.0, 1.0, -1.0), expect.nan_to_num(0.0, 1.0, -1.0)) and torch.equal(torch.isnan(dW[:, 3]).cpu(), torch.isnan(expect))
    c = int((pre[T // 2] > 0).nonzero()[0, 0])
    d = dy.clone()
    d[T // 2, c] = float("inf")
    dx, dW = call(d, x, W)
    rows, cols = [t for t in range(T) if t != T // 2], [n for n in range(N) if n != c]
    assert torch.equal(dx[rows], clean[0][rows]) and torch.equal(dW[cols], clean[1][cols])
    for got, by in ((dx[T // 2], W[c]), (dW[c], x[T // 2])):
        expect = R.d(by) * float("inf")
        assert torch.equal(R.d(got).nan_to_num(0.0, 1.0, -1.0), expect.nan_to_num(0.0, 1.0, -1.0))


@pytest.mark.parametrize("dtype,results", [(BF, "16"), (BF, "32"), (FP, "16"), (FP, "dW32")])
def test_in_a_graph_and_a_workspace_in_use(moe, dtype, results):
    dy, x, W, pre = problem("cut_wide", "swiglu", dtype, seed=4)
    T, N, K = SHAPES["cut_wide"]
    tx, tw = RESULTS[results]
    ws = torch.full((moe.linear_backward_workspace_bytes(T, N, K, "swiglu"),), 255, dtype=torch.uint8, device="cuda")  # NaN of every type
    out = dict(dx=torch.empty(T, K, dtype=tx or dtype, device="cuda"), dW=torch.empty(N, K, dtype=tw or dtype, device="cuda"), db=torch.empty(N, dtype=tw or dtype, device="cuda"))
    expect = [t.clone() for t in moe.linear_backward(dy, x, W, pre=pre, act="swiglu", ws=ws, **out)]
    other = [t.clone() for t in moe.linear_backward(dy * 2, x, W, pre=pre, act="swiglu", ws=ws, **out)]
    held = dy.clone()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        moe.linear_backward(held, x, W, pre=pre, act="swiglu", ws=ws, **out)
    for times, want in ((1, expect), (2, other), (1, expect), (2, other)):
        held.copy_(dy * times)
        for t in out.values():
            t.zero_()
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out.values(), want))


@pytest.mark.parametrize("shape", ["few", "small", "odd", "wide_dx256", "cut"])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_rounded_dz_on_request(moe, shape, dtype):
    dy, x, W, pre = problem(shape, "geglu", dtype, seed=5)
    T, N, K = SHAPES[shape]
    size = moe.linear_backward_workspace_bytes(T, N, K, "geglu", round_dz=True)
    assert size < moe.linear_backward_workspace_bytes(T, N, K, "geglu")
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    got = moe.linear_backward(dy, x, W, pre=pre, act="geglu", bias_grad=True, dx=given(x, F4), grad_dtype=F4, ws=ws, round_dz=True)
    for v, (value, slack), name in zip(got, R.linear_grad(dy, x, W, pre, "geglu", dtype), ("dx", "dW", "db")):
        R.within(v, value, R.stored(value, slack, F4), name)
    with pytest.raises(ValueError, match="workspace"):
        moe.linear_backward(dy, x, W, pre=pre, act="geglu", ws=ws)


def test_no_rows(moe):
    x, W, e = torch.empty(0, 16, dtype=FP, device="cuda"), torch.ones(8, 16, dtype=FP, device="cuda"), torch.empty(0, 8, dtype=FP, device="cuda")
    for act, dy in (("silu", e), ("swiglu", e[:, :4])):
        dx, dW, db = moe.linear_backward(dy, x, W, pre=e, act=act, bias_grad=True, grad_dtype=F4)
        assert dx.shape == (0, 16) and (dW == 0).all() and (db == 0).all()


@pytest.mark.parametrize("act", ["silu", "gelu", "geglu"])
@pytest.mark.parametrize("T", [1, 70])
def test_parts_add_up(moe, T, act):
    """With ones for weights and inputs the three bf16 parts give dz itself, to the last bit, which db shows: of one row, and of rows of zeros beside it.
    Values from 2^-90 to 2^90, those of few bits among them."""
    N = 512
    g = torch.Generator().manual_seed(6)
    cols = N // 2 if act in R.GATED else N
    dy = torch.zeros(T, cols, dtype=BF, device="cuda")
    dy[T // 2] = rnd(g, cols) * (2.0 ** torch.randint(-90, 90, (cols,), generator=g)).to(BF).cuda()
    dy[T // 2, :cols // 4] = (2.0 ** torch.randint(-90, 90, (cols // 4,), generator=g)).to(BF).cuda()
    pre = rnd(g, T, N)
    W, x = torch.eye(N, dtype=BF, device="cuda"), torch.ones(T, 8, dtype=BF, device="cuda")
    dx, _, db = moe.linear_backward(dy, torch.zeros(T, N, dtype=BF, device="cuda"), W, pre=pre, act=act, bias_grad=True, dx=torch.empty(T, N, device="cuda"), grad_dtype=F4)
    assert torch.equal(dx[T // 2], db) and (db != 0).all()
    assert (dx[:T // 2] == 0).all() and (dx[T // 2 + 1:] == 0).all()
    _, dW, _ = moe.linear_backward(dy, x, None, pre=pre, act=act, dx=False, grad_dtype=F4)
    assert torch.equal(dW, db[:, None].expand(N, 8))
    # two parts: 2^-15 of dz, and the result's own rounding
    for dtype in (BF, FP):
        e = torch.where(torch.arange(cols) % 2 == 0, 1.0, 2.0 ** -6).cuda()
        d = torch.zeros(T, cols, dtype=dtype, device="cuda")
        d[T // 2] = (rnd(g, cols, dtype=F4) * e).to(dtype)
        dx, _, db = moe.linear_backward(d, torch.zeros(T, N, dtype=dtype, device="cuda"), W.to(dtype), pre=pre.to(dtype), act=act, bias_grad=True)
        _, _, db = moe.linear_backward(d, None, W.to(dtype), pre=pre.to(dtype), act=act, dx=False, dW=False, bias_grad=True, grad_dtype=F4)
        value = R.d(db)
        R.within(dx[T // 2], value, R.stored(value, 2.0 ** -15 * value.abs() if dtype is BF else 2.0 ** -22 * value.abs() + 2.0 ** -25, dtype), "dx")
