"""Low-rank adapters beside a shared projection and their gradients on the GPU
against plain 64-bit forms, element by element."""
import pytest
import torch

import grouped_reference as R
from test_gpu_grouped import BF, F4, FP, gen, moe, rnd, strided  # noqa: F401

pytestmark = pytest.mark.gpu


def batch(kind, T, n, g):
    """Adapter of each row: outside [0, n) is none."""
    if kind == "runs":
        ids = torch.sort(torch.randint(0, n, (T,), generator=g)).values
    elif kind == "one":
        ids = torch.full((T,), n - 1)
    elif kind == "none":
        ids = torch.full((T,), -1)
    else:
        ids = torch.randint(-1, n + 1, (T,), generator=g)
    return ids.to(torch.int32).cuda()


@pytest.mark.parametrize("T,n", [(1, 1), (1, 1024), (64, 7), (1000, 3), (1024, 1024), (1025, 64), (5000, 1), (16384, 300), (0, 5)])
@pytest.mark.parametrize("kind", ["mixed", "runs", "none"])
def test_plan(moe, T, n, kind):  # noqa: F811
    ids = batch(kind, T, n, gen(T + n))
    rows, offsets = moe.adapter_plan(ids, n)
    key = torch.where((ids >= 0) & (ids < n), ids, n).cpu()
    assert torch.equal(rows.cpu(), torch.sort(key, stable=True).indices.to(torch.int32))
    counts = torch.bincount(key, minlength=n + 1)[:n]
    assert torch.equal(offsets.cpu()[1:], counts.cumsum(0).to(torch.int32)) and int(offsets[0]) == 0


#         T, n, K, N, r
SIZES = [(1, 1, 64, 64, 16), (1, 3, 2048, 2048, 16), (3, 2, 8, 8, 1), (33, 4, 200, 136, 8), (64, 64, 256, 512, 16), (70, 5, 77, 131, 5),
         (100, 2, 130, 67, 17), (257, 3, 512, 72, 33), (90, 2, 64, 264, 64), (65, 2, 136, 128, 100), (40, 2, 96, 1100, 128), (300, 1, 1, 1, 2)]


def problem(T, n, K, N, r, dtype, kind="mixed"):
    g = gen(T + n + K + r)
    ids = batch(kind, T, n, g)
    x, dy = rnd(g, T, K, dtype=dtype), rnd(g, T, N, dtype=dtype)
    A, B = rnd(g, n, r, K, dtype=dtype, scale=K ** -0.5), rnd(g, n, N, r, dtype=dtype, scale=r ** -0.5)
    return g, ids, x, dy, A, B, (torch.rand(n, generator=g) + 0.5).cuda()


@pytest.mark.parametrize("T,n,K,N,r", SIZES)
@pytest.mark.parametrize("dtype,out", [(BF, BF), (FP, F4), (BF, F4), (FP, FP)])
def test_forward(moe, T, n, K, N, r, dtype, out):  # noqa: F811
    for kind in ("mixed", "runs"):
        g, ids, x, _, A, B, scale = problem(T, n, K, N, r, dtype, kind)
        plan = moe.adapter_plan(ids, n)
        xs = strided(x, 8, float("nan"))[1]
        wide, base = strided(rnd(g, T, N, dtype=out), 8, 2.0)
        value, slack, _, _ = R.adapter(x, A, B, scale, ids, base)
        y = moe.adapter_forward(xs, A, B, scale, plan, base=base)
        assert y.dtype == out
        R.within(y, value, R.stored(value, slack, out), "y")
        moe.adapter_forward(xs, A, B, scale, plan, base=base, out=base)  # in place, strided
        assert torch.equal(base, y) and (wide[:, N:] == 2.0).all()
        value, slack, _, _ = R.adapter(x, A, B, None, ids, None)
        y = moe.adapter_forward(x, A, B, None, plan, out_dtype=out)
        R.within(y, value, R.stored(value, slack, out), "y without base and scale")


@pytest.mark.parametrize("T,n,K,N,r", SIZES)
@pytest.mark.parametrize("dtype,grads", [(BF, BF), (FP, F4), (BF, F4)])
def test_gradients(moe, T, n, K, N, r, dtype, grads):  # noqa: F811
    for kind in ("mixed", "one"):
        g, ids, x, dy, A, B, scale = problem(T, n, K, N, r, dtype, kind)
        plan = moe.adapter_plan(ids, n)
        start = rnd(g, T, K, dtype=grads)
        want = R.adapter_grad(dy, x, A, B, scale, ids, start)
        got = moe.adapter_backward(strided(dy, 8, float("nan"))[1], strided(x, 8, float("nan"))[1], A, B, scale, plan, dx_base=start, grad_dtype=grads)
        for name, t, (value, slack) in zip(("dx", "dA", "dB"), got, want):
            R.within(t, value, R.stored(value, slack, t.dtype), name)
        dx = start.clone()
        moe.adapter_backward(dy, x, A, B, scale, plan, dx_base=dx, dx=dx)
        assert torch.equal(dx, got[0])
        if grads == F4:
            dA, dB = rnd(g, n, r, K, dtype=F4), rnd(g, n, N, r, dtype=F4)
            a0, b0 = R.d(dA), R.d(dB)
            moe.adapter_backward(dy, x, A, B, scale, plan, dA=dA, dB=dB, accumulate=True)
            for name, t, s, (value, slack) in zip(("dA", "dB"), (dA, dB), (a0, b0), want[1:]):
                R.within(t, value + s, R.stored(value + s, slack + 2 * R.U * s.abs(), F4), name + " added")
        dx = moe.adapter_backward(dy, x, A, B, None, plan)[0]
        value, slack = R.adapter_grad(dy, x, A, B, None, ids, None)[0]
        R.within(dx, value, R.stored(value, slack, dtype), "dx without base and scale")


# 8 to 24 rows an adapter (32 rows a workgroup), many an adapter (rows shared by the waves), a long batch
FORMS = [(60, 4, 136, 200, 20), (61, 4, 77, 131, 30), (60, 4, 136, 200, 40), (62, 5, 130, 67, 64), (300, 2, 72, 136, 16),
         (280, 2, 77, 40, 24), (300, 2, 136, 72, 50), (290, 2, 64, 131, 128), (16400, 3, 16, 24, 9), (4100, 9, 24, 16, 36)]


@pytest.mark.parametrize("T,n,K,N,r", FORMS)
@pytest.mark.parametrize("dtype,out", [(BF, F4), (FP, FP)])
def test_forms(moe, T, n, K, N, r, dtype, out):  # noqa: F811
    test_forward(moe, T, n, K, N, r, dtype, out)
    test_gradients(moe, T, n, K, N, r, dtype, out)


@pytest.mark.parametrize("kind", ["mixed", "one"])
def test_gradients_against_differences(moe, kind):  # noqa: F811
    """y is linear in x, in A and in B: <y, G> changes by the gradient times the change."""
    T, n, K, N, r = 60, 3, 128, 96, 12
    g, ids, x, dy, A, B, scale = problem(T, n, K, N, r, BF, kind)
    plan = moe.adapter_plan(ids, n)
    loss = lambda *a: float((R.d(moe.adapter_forward(*a, scale, plan, out_dtype=F4)) * R.d(dy)).sum())  # noqa: E731
    grads = moe.adapter_backward(dy, x, A, B, scale, plan, dx=torch.empty(T, K, dtype=F4, device="cuda"), grad_dtype=F4)
    args = [x, A, B]
    bound = R.adapter_grad(dy, x, A, B, scale, ids, None)
    for i, (grad, (_, gs)) in enumerate(zip(grads, bound)):
        other = list(args)
        other[i] = rnd(g, *args[i].shape, scale=0.1)
        change = R.d(other[i]) - R.d(args[i])
        slack = float((gs * change.abs()).sum()) + R.U * float((R.d(grad) * change).abs().sum())
        for a in (args, other):
            y, s, _, _ = R.adapter(*a, scale, ids, None)
            slack += float(((s + R.U * y.abs()) * R.d(dy).abs()).sum())
        assert abs(loss(*other) - loss(*args) - float((R.d(grad) * change).sum())) <= slack, i


def test_rows_without_adapter_and_bad_rows(moe):  # noqa: F811
    g, ids, x, dy, A, B, scale = problem(50, 3, 64, 48, 8, BF, "none")
    plan = moe.adapter_plan(ids, 3)
    base = rnd(g, 50, 48)
    base[3, 4] = float("nan")
    y = moe.adapter_forward(x, A, B, scale, plan, base=base)
    assert torch.equal(y.view(torch.int16), base.view(torch.int16))
    assert (moe.adapter_forward(x, A, B, scale, plan) == 0).all()
    dx, dA, dB = moe.adapter_backward(dy, x, A, B, scale, plan)
    assert (dx == 0).all() and (dA == 0).all() and (dB == 0).all()
    # entries of rows outside the batch are skipped
    ids = torch.zeros(50, dtype=torch.int32, device="cuda")
    rows, offsets = moe.adapter_plan(ids, 3)
    rows[7], rows[8] = -1, 50
    y = torch.full((50, 48), 9.0, dtype=BF, device="cuda")
    moe.adapter_forward(x, A, B, scale, (rows, offsets), out=y)
    keep = torch.ones(50, dtype=torch.bool, device="cuda")
    keep[7:9] = False
    want = moe.adapter_forward(x, A, B, scale, moe.adapter_plan(ids, 3))
    assert torch.equal(y[keep], want[keep]) and (y[7:9] == 9.0).all()


def test_nan_stays_in_its_row(moe):  # noqa: F811
    g, ids, x, dy, A, B, scale = problem(70, 2, 72, 40, 8, BF, "mixed")
    plan = moe.adapter_plan(ids, 2)
    want = moe.adapter_forward(x, A, B, scale, plan)
    dx = moe.adapter_backward(dy, x, A, B, scale, plan)[0]
    hit = int((ids == 1).nonzero()[0, 0])
    x2, dy2 = x.clone(), dy.clone()
    x2[hit, 5], dy2[hit, 6] = float("nan"), float("inf")
    y = moe.adapter_forward(x2, A, B, scale, plan)
    dx2, dA, dB = moe.adapter_backward(dy2, x2, A, B, scale, plan)
    others = torch.arange(70, device="cuda") != hit
    assert torch.equal(y[others], want[others]) and torch.equal(dx2[others], dx[others])
    assert torch.isfinite(dA[0]).all() and torch.isfinite(dB[0]).all() and not torch.isfinite(dA[1]).all()


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("r", [1, 5, 16, 17, 40, 100])
def test_infinities_keep_their_sign(moe, dtype, r):  # noqa: F811
    """An infinite row gives the formula's infinities; ranks that only fill up the
    kernel's tiles (0 times infinity) have no part in it."""
    g, ids, x, dy, A, B, scale = problem(70, 2, 72, 40, r, dtype, "mixed")
    A, B, scale = A.abs() + 0.5, B.abs() + 0.5, scale.abs() + 0.5
    plan = moe.adapter_plan(ids, 2)
    hit = int((ids == 1).nonzero()[0, 0])
    x[hit, 5], dy[hit, 6] = float("inf"), float("-inf")
    assert (moe.adapter_forward(x, A, B, scale, plan)[hit] == float("inf")).all()
    assert (moe.adapter_backward(dy, x, A, B, scale, plan)[0][hit] == float("-inf")).all()


def test_beside_the_int4_projection(moe):  # noqa: F811
    """A serving step: the shared int4 projection, then the adapters in place on
    its fp32 result; equal to adding them to a copy."""
    from synth import moe_inputs as S
    import numpy as np
    T, n, K, N, r = 40, 4, 256, 256, 16
    p = S.make_custom(T, S.LayerShape(d=256, f=128, E=1, k=1, f_sh=128), seed=2)
    up = lambda a, t: torch.from_numpy(np.ascontiguousarray(a).view(t)).cuda()  # noqa: E731
    Wq, Ws, Wb = (up(p.layer["sh_gu_q"], np.int32), *(up(p.layer[k], np.int16).view(BF) for k in ("sh_gu_s", "sh_gu_b")))
    g, ids, x, _, A, B, scale = problem(T, n, K, N, r, BF)
    rt = moe.route(torch.zeros(T, 1, device="cuda"), 1)
    y = torch.empty(T, N, device="cuda")
    moe.grouped_gemm_int4(x, None, N, K, Wq, Ws, Wb, rt["block_map"], rt["num_blocks"], y)
    value, slack, _, _ = R.adapter(x, A, B, scale, ids, y)
    moe.adapter_forward(x, A, B, scale, moe.adapter_plan(ids, n), base=y, out=y)
    R.within(y, value, R.stored(value, slack, F4), "y")


def test_captured_and_replayed(moe):  # noqa: F811
    T, n, K, N, r = 90, 4, 136, 72, 16
    g, ids, x, dy, A, B, scale = problem(T, n, K, N, r, BF)

    def step():
        plan = moe.adapter_plan(ids, n)
        return (moe.adapter_forward(x, A, B, scale, plan), *moe.adapter_backward(dy, x, A, B, scale, plan))

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for i in range(4):
        ids.copy_(batch("mixed" if i % 2 else "runs", T, n, gen(i)))
        x.copy_(rnd(gen(40 + i), T, K))
        want = [t.clone() for t in step()]
        for t in held:
            t.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, want)), f"replay {i}"


def test_refused_tensors(moe):  # noqa: F811
    g, ids, x, dy, A, B, scale = problem(8, 2, 16, 24, 4, BF)
    plan = moe.adapter_plan(ids, 2)
    bad = [(TypeError, lambda: moe.adapter_forward(x, A.half(), B, scale, plan)), (ValueError, lambda: moe.adapter_forward(x, A, B[:1], scale, plan)),
           (ValueError, lambda: moe.adapter_forward(x, A, B, scale[:1], plan)), (TypeError, lambda: moe.adapter_forward(x, A, B, scale.double(), plan)),
           (ValueError, lambda: moe.adapter_forward(x[:4], A, B, scale, plan)), (ValueError, lambda: moe.adapter_plan(ids, 0)),
           (TypeError, lambda: moe.adapter_forward(x, A, B, scale, plan, base=torch.zeros(8, 24, device="cuda"), out_dtype=BF)),
           (ValueError, lambda: moe.adapter_backward(dy, x, A, B, scale, plan, accumulate=True)),
           (ValueError, lambda: moe.adapter_backward(dy, x, A, B, scale, plan, ws=torch.empty(16, dtype=torch.uint8, device="cuda"))),
           (ValueError, lambda: moe.adapter_backward(dy, x, A, B, scale, plan, ws=torch.empty(1, dtype=torch.uint8, device="cuda").expand(1 << 16))),
           (TypeError, lambda: moe.adapter_plan(ids.long(), 2))]
    for kind, f in bad:
        with pytest.raises(kind):
            f()
